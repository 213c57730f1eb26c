"""What is measured of the operators by which every token picks its weights:
routing to experts, the way into expert order and back, and low-rank adapters
of many requests beside a shared projection.

  route     scores s = softmax or sigmoid of the logits [T,E]; experts ranked by
            s + bias (without a bias by the logits), among those of the best
            groups only; the topk first, their weights s, renormalised, scaled
  dispatch  the rows of x [T,K], and their scales, copied to where the experts'
            product wants them: expert by expert, by token within one; offsets
            per expert and each choice's row (-1: another GPU's expert, or none)
  combine   out[t] = base[t] + sum_j weights[t,j] * rows[slots[t,j]]
  adapters  out[t] = y[t] + scales[a] * B[a] (A[a] x[t]), a = adapters[t], -1: none

`run` takes the inputs that `prepare` makes through one of them: by elementary
operations in 32 bits where `own` is false (in 64 where experts are compared),
by the calls of block_scaled_fp8_gemm_amd where it is true.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "fp8": 1}


def listed():
    return [
        # One token of a decoder: a single row of scores.
        {"name": "route_token", "op": "route", "T": 1, "E": 256, "topk": 8, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "group_score": "max", "dtype": "bf16", "masked": 0.0},
        # A decode batch: sigmoid scores with a bias for balance, 4 of 8 groups by their two best.
        {"name": "route_decode", "op": "route", "T": 64, "E": 256, "topk": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_score": "top2", "dtype": "fp32", "masked": 0.0},
        # A padded batch over a number of experts that no wave divides.
        {"name": "route_odd", "op": "route", "T": 777, "E": 60, "topk": 6, "score": "softmax", "bias": False,
         "groups": 1, "topk_groups": 1, "group_score": "max", "dtype": "fp16", "masked": 0.2},
        # The same scores as the decode batch's for the tokens of a prefill.
        {"name": "route_prefill", "op": "route", "T": 16384, "E": 256, "topk": 8, "score": "sigmoid", "bias": True,
         "groups": 8, "topk_groups": 4, "group_score": "top2", "dtype": "fp32", "masked": 0.0},
        # The int8 codes of a decode batch for 8 of 256 experts per token.
        {"name": "dispatch_decode", "op": "dispatch", "T": 64, "E": 256, "local": 256, "topk": 8, "K": 4096,
         "kind": "int8", "skew": 0.0},
        # Half of 64 experts on this GPU, bf16 rows of an odd width, uneven loads.
        {"name": "dispatch_share", "op": "dispatch", "T": 1001, "E": 64, "local": 32, "topk": 6, "K": 1027,
         "kind": "bf16", "skew": 0.5},
        # A prefill's codes.
        {"name": "dispatch_prefill", "op": "dispatch", "T": 4096, "E": 256, "local": 256, "topk": 8, "K": 4096,
         "kind": "int8", "skew": 0.0},
        # The way back for a decode batch, and for a prefill beside the shared expert's output.
        {"name": "combine_decode", "op": "combine", "T": 64, "topk": 8, "D": 4096, "dtype": "bf16", "out": "bf16",
         "base": False, "dropped": 0.0},
        {"name": "combine_prefill", "op": "combine", "T": 4096, "topk": 8, "D": 4096, "dtype": "bf16", "out": "bf16",
         "base": True, "dropped": 0.0},
        # 64 requests of one token each over 16 adapters beside a square projection.
        {"name": "adapters_decode", "op": "adapters", "T": 64, "requests": 64, "L": 16, "R": 16, "K": 4096, "N": 4096,
         "dtype": "bf16", "out": "bf16", "bare": 0.1},
        # A few prompts with sizes that no tile divides, 32-bit outputs.
        {"name": "adapters_odd", "op": "adapters", "T": 301, "requests": 5, "L": 3, "R": 10, "K": 1000, "N": 1537,
         "dtype": "fp16", "out": "fp32", "bare": 0.2},
        # A prefill of several prompts.
        {"name": "adapters_prefill", "op": "adapters", "T": 16384, "requests": 12, "L": 16, "R": 16, "K": 4096,
         "N": 4096, "dtype": "bf16", "out": "bf16", "bare": 0.1},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _size(rng, lo, hi, unit):
    """Half of the sizes are any number, the others a multiple of `unit`."""
    v = _log(rng, lo, hi)
    return v if rng.random() < 0.5 else max(unit, v // unit * unit)


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "adapters"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 8, 256 // groups)
        topk_groups = rng.randint(1, groups)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "topk": rng.randint(1, min(8, E // groups)),
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "groups": groups,
                "topk_groups": topk_groups, "group_score": rng.choice(["max", "top2"]),
                "dtype": rng.choice(["bf16", "fp16", "fp32"]), "masked": rng.choice([0.0, 0.0, 0.3])}
    if op == "dispatch":
        E = _log(rng, 8, 256)
        topk, K, kind = rng.randint(1, 8), _size(rng, 64, 4096, 128), rng.choice(["int8", "fp8", "bf16"])
        K = K if kind != "fp8" else max(128, K // 128 * 128)
        T = min(_log(rng, 1, 4096), (4096 * 4096 * 8) // (topk * K * SIZES[kind] * (3 if kind == "fp8" else 1)))
        return {"op": op, "T": T, "E": E, "local": rng.choice([E, max(1, E // 2)]), "topk": topk, "K": K,
                "kind": kind, "skew": round(rng.uniform(0.0, 0.6), 2)}
    if op == "combine":
        topk, D = rng.randint(1, 8), _size(rng, 32, 8192, 128)
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        return {"op": op, "T": min(_log(rng, 1, 4096), (4096 * 4096 * 8 * 2) // (topk * D * SIZES[dtype])),
                "topk": topk, "D": D, "dtype": dtype, "out": rng.choice([dtype, "fp32"]),
                "base": rng.random() < 0.5, "dropped": rng.choice([0.0, 0.0, 0.5])}
    L, R, K, N = _log(rng, 1, 64), _size(rng, 4, 128, 8), _size(rng, 64, 4096, 128), _size(rng, 64, 4096, 128)
    L = max(1, min(L, 1024 // R))
    T = min(_log(rng, 1, 16384), (16384 * 256 * 8192) // (L * R * (K + N)))
    return {"op": op, "T": T, "requests": min(T, _log(rng, 1, 256)), "L": L, "R": R, "K": K, "N": N,
            "dtype": rng.choice(["bf16", "fp16"]), "out": rng.choice(["bf16", "fp16", "fp32"]),
            "bare": rng.choice([0.0, 0.1, 0.5])}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _picked(g, T, E, topk, skew):
    """topk different experts for each token, some experts more popular than others."""
    noise = -torch.log(-torch.log(_uniform(g, T, E).clamp_(1e-6, 1 - 1e-6)))
    return torch.topk(skew * _normal(g, E) + noise, topk, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, T = case["op"], case["T"]
    s = {"case": case, "op": op}
    if op == "route":
        E = case["E"]
        # Experts differ in popularity; the bias works against that, as it is trained to.
        popular = 0.5 * _normal(g, E)
        s["logits"] = (1.5 * _normal(g, T, E) + popular).to(DTYPES[case["dtype"]])
        s["bias"] = -0.05 * popular if case["bias"] else None
        s["mask"] = _uniform(g, T) < case["masked"] if case["masked"] else None
        s["scale"] = 2.5 if case["score"] == "sigmoid" else 1.0
    elif op == "dispatch":
        E, K = case["E"], case["K"]
        s["first"] = (E - case["local"]) // 2
        s["experts"] = _picked(g, T, E, min(case["topk"], E), case["skew"])
        x = _normal(g, T, K)
        if case["kind"] == "bf16":
            s["x"], s["x_scale"], scales = x.to(torch.bfloat16), None, None
        elif case["kind"] == "int8":
            s["x"], scales = x.mul_(127.0 / 4.0).round_().clamp_(-127, 127).to(torch.int8), ()
        else:
            s["x"], scales = x.mul_(448.0 / 4.0).clamp_(-448, 448).to(torch.float8_e4m3fn), (K // 128,)
        n = s["experts"].numel()
        # The rows and scales in expert order; what no expert here takes is left as it is.
        s["rows"] = torch.zeros(n, K, device="cuda", dtype=s["x"].dtype)
        s["row_scale"] = None
        if scales is not None:
            s["x_scale"] = 0.01 + 0.01 * _uniform(g, T, *scales)
            s["row_scale"] = torch.zeros(n, *scales, device="cuda")
    elif op == "combine":
        topk, D = case["topk"], case["D"]
        n = T * topk
        s["slots"] = torch.randperm(n, generator=g, device="cuda", dtype=torch.int32).view(T, topk)
        if case["dropped"]:
            s["slots"] = torch.where(_uniform(g, T, topk) < case["dropped"], -1, s["slots"])
        s["rows"] = _normal(g, n, D).to(DTYPES[case["dtype"]])
        s["weights"] = 2.5 * torch.softmax(_normal(g, T, topk), dim=1)
        s["base"] = _normal(g, T, D).to(DTYPES[case["dtype"]]) if case["base"] else None
    else:
        L, R, K, N = case["L"], case["R"], case["K"], case["N"]
        t = DTYPES[case["dtype"]]
        s["x"] = _normal(g, T, K).to(t)
        s["y"] = _normal(g, T, N).to(DTYPES[case["out"]])
        s["A"] = (_normal(g, L, R, K) / K ** 0.5).to(t)
        s["B"] = (0.3 * _normal(g, L, N, R) / R ** 0.5).to(t)
        s["scales"] = 1.0 + _uniform(g, L)
        # Requests are runs of tokens, a share of them without an adapter.
        starts = torch.zeros(T, device="cuda", dtype=torch.int64)
        starts[torch.randperm(T, generator=g, device="cuda")[:case["requests"]]] = 1
        chosen = torch.randint(0, L, (T + 1,), generator=g, device="cuda", dtype=torch.int32)
        chosen = torch.where(_uniform(g, T + 1) < case["bare"], -1, chosen)
        s["adapters"] = chosen[starts.cumsum(0)].contiguous()
    return s


# ---------------------------------------------------------------------------
# The plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _plain_route(s):
    c, bias = s["case"], s["bias"]
    logits = s["logits"].double()   # scores that lie next to one another are told apart
    T, E = logits.shape
    score = torch.sigmoid(logits) if c["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    rank = logits if bias is None else score + bias.double()
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices
    if c["groups"] > 1:
        if c["group_score"] == "max":
            best = rank.view(T, c["groups"], -1).amax(dim=2)
        else:
            value = score if bias is None else rank
            best = torch.sort(value.view(T, c["groups"], -1), dim=2, descending=True).values[..., :2].sum(dim=2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        out = torch.ones(T, c["groups"], device="cuda", dtype=torch.int8).scatter_(1, kept, 0)
        out = out.gather(1, order // (E // c["groups"]))
        order = order.gather(1, torch.sort(out, dim=1, stable=True).indices)
    experts = order[:, :c["topk"]]
    weights = score.gather(1, experts).float()
    weights = weights / weights.sum(dim=1, keepdim=True).clamp(min=1e-20) * s["scale"]
    if s["mask"] is not None:
        weights = torch.where(s["mask"][:, None], 0.0, weights)
        experts = torch.where(s["mask"][:, None], -1, experts)
    return weights, experts.to(torch.int32)


def _plain_dispatch(s):
    E, n = s["case"]["local"], s["experts"].numel()
    e = s["experts"].reshape(-1) - s["first"]
    here = (e >= 0) & (e < E)
    order = torch.sort(torch.where(here, e, E), stable=True).indices
    offsets = (e[None, :] < torch.arange(1, E + 1, device="cuda", dtype=torch.int32)[:, None]) & here
    offsets = torch.cat([e.new_zeros(1), offsets.sum(dim=1, dtype=torch.int32)])
    at = torch.arange(n, device="cuda", dtype=torch.int32)
    slots = torch.empty_like(e)
    slots[order] = at
    slots = torch.where(here, slots, -1).view(s["experts"].shape)
    token = order // s["experts"].shape[1]
    filled = at < offsets[-1]

    def moved(x):   # E4M3 codes move as bytes
        b = x.view(torch.int8) if x.dtype == torch.float8_e4m3fn else x
        b = torch.where(filled.view(-1, *[1] * (x.dim() - 1)), b[token], torch.zeros((), device="cuda", dtype=b.dtype))
        return b.view(x.dtype)

    return moved(s["x"]), None if s["x_scale"] is None else moved(s["x_scale"]), offsets, slots


def _plain(s):
    if s["op"] == "route":
        return _plain_route(s)
    if s["op"] == "dispatch":
        rows, scale, offsets, slots = _plain_dispatch(s)
        return _values(rows), scale, offsets, slots
    if s["op"] == "combine":
        w = torch.where(s["slots"] >= 0, s["weights"], 0.0)
        out = (s["rows"].float()[s["slots"].clamp(min=0)] * w[..., None]).sum(dim=1)
        return (out if s["base"] is None else out + s["base"].float()).to(DTYPES[s["case"]["out"]])
    # All adapters' first products, those of other adapters' columns zeroed, and all second ones at once.
    L, R, K = s["A"].shape
    share = torch.where(s["adapters"][:, None] == torch.arange(L, device="cuda", dtype=torch.int32), s["scales"], 0.0)
    h = (s["x"].float() @ s["A"].view(L * R, K).float().t()).view(-1, L, R) * share[..., None]
    d = h.view(-1, L * R) @ s["B"].transpose(1, 2).reshape(L * R, -1).float()
    return (s["y"].float() + d).to(s["y"].dtype)


def _values(rows):
    """E4M3 codes as the values that they stand for, beside their scales."""
    return rows.to(torch.bfloat16) if rows.dtype == torch.float8_e4m3fn else rows


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    import block_scaled_fp8_gemm_amd as fbg

    c = s["case"]
    if s["op"] == "route":
        return fbg.route_experts(s["logits"], c["topk"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                 topk_groups=c["topk_groups"], group_score=c["group_score"], renormalize=True,
                                 scale=s["scale"], mask=s["mask"])
    if s["op"] == "dispatch":
        rows, scale, offsets, slots = fbg.dispatch_tokens(s["experts"], c["local"], s["x"], s["x_scale"],
                                                          first_expert=s["first"], rows=s["rows"],
                                                          row_scale=s["row_scale"])
        return _values(rows), scale, offsets, slots
    if s["op"] == "combine":
        return fbg.combine_experts(s["rows"], s["slots"], s["weights"], base=s["base"], out_dtype=DTYPES[c["out"]])
    return fbg.add_adapters(s["y"], s["x"], s["A"], s["B"], s["adapters"], s["scales"], out=torch.empty_like(s["y"]))


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        def lowest_best(value, allowed):
            """The place of each row's largest allowed value, the lowest of equals."""
            v = torch.where(allowed, value, -math.inf)
            at = torch.arange(v.shape[1], device="cuda").expand_as(v)
            return torch.where(allowed & (v == v.max(dim=1, keepdim=True).values), at, v.shape[1]).min(dim=1).values

        z = s["logits"].double()
        T, E = z.shape
        if case["score"] == "sigmoid":
            score = 1 / (1 + torch.exp(-z))
        else:
            score = torch.exp(z - z.max(dim=1, keepdim=True).values)
            score = score / score.sum(dim=1, keepdim=True)
        rank = z if s["bias"] is None else score + s["bias"].double()
        row = torch.arange(T, device="cuda")
        allowed = torch.ones(T, E, dtype=torch.bool, device="cuda")
        if case["groups"] > 1:
            size = E // case["groups"]
            value = rank if case["group_score"] == "max" or s["bias"] is not None else score
            best = torch.zeros(T, case["groups"], dtype=torch.float64, device="cuda")
            for i in range(case["groups"]):
                top = value[:, i * size:(i + 1) * size].topk(min(2 if case["group_score"] == "top2" else 1, size), dim=1)
                best[:, i] = top.values.sum(dim=1)
            allowed[:] = False
            left = torch.ones(T, case["groups"], dtype=torch.bool, device="cuda")
            for _ in range(case["topk_groups"]):
                i = lowest_best(best, left)
                left[row, i] = False
                allowed |= (torch.arange(E, device="cuda") // size)[None, :] == i[:, None]
        experts = torch.zeros(T, case["topk"], dtype=torch.int64, device="cuda")
        for j in range(case["topk"]):
            experts[:, j] = lowest_best(rank, allowed)
            allowed[row, experts[:, j]] = False
        weights = score.gather(1, experts)
        weights = weights / weights.sum(dim=1, keepdim=True).clamp(min=1e-20) * s["scale"]
        if s["mask"] is not None:
            weights[s["mask"]] = 0.0
            experts[s["mask"]] = -1
        return weights, experts.to(torch.int32)
    if s["op"] == "dispatch":
        experts = s["experts"].cpu() - s["first"]
        topk = experts.shape[1]
        rows, scale, slots, ends = s["rows"], s["row_scale"], torch.full_like(experts, -1), [0]
        flat = experts.reshape(-1)
        for e in range(case["local"]):
            mine = (flat == e).nonzero()[:, 0]
            lo, hi = ends[-1], ends[-1] + len(mine)
            slots.view(-1)[mine] = torch.arange(lo, hi, dtype=torch.int32)
            token = (mine // topk).cuda()
            rows.view(torch.uint8)[lo:hi] = s["x"].view(torch.uint8)[token]
            if scale is not None:
                scale[lo:hi] = s["x_scale"][token]
            ends.append(hi)
        return _values(rows), scale, torch.tensor(ends, dtype=torch.int32, device="cuda"), slots.cuda()
    if s["op"] == "combine":
        out = torch.zeros(case["T"], case["D"], dtype=torch.float64, device="cuda")
        if s["base"] is not None:
            out += s["base"]
        for j in range(case["topk"]):
            t = (s["slots"][:, j] >= 0).nonzero()[:, 0]
            out[t] += s["rows"][s["slots"][t, j]].double() * s["weights"][t, j, None].double()
        return out
    out = s["y"].double()
    for a in range(case["L"]):
        t = (s["adapters"] == a).nonzero()[:, 0]
        if len(t):
            h = torch.matmul(s["x"][t].double(), s["A"][a].double().t().contiguous())
            out[t] += torch.matmul(h, s["B"][a].double().t().contiguous()) * s["scales"][a].double()
    return out


def work(case):
    """Bytes (each input read once, each output written once) and operations
    of one pass."""
    op, T = case["op"], case["T"]
    if op == "route":
        E, topk = case["E"], case["topk"]
        return {"bytes": T * E * SIZES[case["dtype"]] + T * topk * 8 + (4 * E if case["bias"] else 0)
                + (T if case["masked"] else 0), "flops": 5 * T * E}
    if op == "dispatch":
        K, topk = case["K"], min(case["topk"], case["E"])
        row = K * SIZES[case["kind"]] + {"bf16": 0, "int8": 4, "fp8": K // 32}[case["kind"]]
        placed = T * topk * case["local"] / case["E"]
        return {"bytes": T * row + placed * row + T * topk * 8 + 4 * (case["local"] + 1), "flops": 0}
    if op == "combine":
        topk, D, size = case["topk"], case["D"], SIZES[case["dtype"]]
        placed = T * topk * (1 - case["dropped"])
        return {"bytes": placed * D * size + T * topk * 8 + (T * D * size if case["base"] else 0)
                + T * D * SIZES[case["out"]], "flops": 2 * placed * D}
    L, R, K, N = case["L"], case["R"], case["K"], case["N"]
    used, busy = T * (1 - case["bare"]), L * (1 - (1 - (1 - case["bare"]) / L) ** case["requests"])
    return {"bytes": used * K * 2 + busy * R * (K + N) * 2 + 2 * T * N * SIZES[case["out"]] + 4 * T,
            "flops": 2 * used * R * (K + N)}
