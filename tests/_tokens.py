"""Plain 64-bit forms, on the CPU, of the operators by which every token picks
its weights, and how far an fp32 evaluation may be from them (U32, U_OUT, TINY:
the unit roundoffs and half subnormal steps of tests._int8)."""
import numpy as np
import torch

from tests._int8 import DTYPES, TINY, U32, U_OUT  # noqa: F401


def route(logits, topk, score="softmax", bias=None, groups=1, topk_groups=1, group_score="max", renormalize=True,
          scale=1.0, mask=None):
    """(weights in 64 bits, experts, tol): see fbg_route_experts."""
    z = logits.double().numpy()
    T, E = z.shape
    b = None if bias is None else bias.double().numpy()
    weights, experts, tol = np.zeros((T, topk)), np.full((T, topk), -1, np.int32), np.zeros((T, topk))
    for t in range(T):
        if mask is not None and bool(mask[t]):
            continue
        row = z[t]
        off = np.isnan(row).any() or (row == np.inf).any()
        if b is not None:
            off = off or np.isnan(b).any() or (b == np.inf).any()
        if off or (score == "softmax" and row.max() == -np.inf):
            weights[t], experts[t] = np.nan, np.arange(topk)
            continue
        with np.errstate(over="ignore"):
            if score == "softmax":
                s = np.exp(row - row.max())
                s /= s.sum()
                far = row.max() - row
            else:
                s = 1 / (1 + np.exp(-row))
                far = np.abs(row)
        c = row if b is None else s + b
        order = np.argsort(-c, kind="stable")
        if groups > 1:
            v = (c if group_score == "max" or b is not None else s).reshape(groups, -1)
            best = np.sort(v, axis=1)[:, ::-1]
            best = best[:, 0] if group_score == "max" else best[:, :2].sum(axis=1)
            kept = np.argsort(-best, kind="stable")[:topk_groups]
            order = order[np.isin(order // (E // groups), kept)]
        e = order[:topk]
        w = s[e]
        if renormalize:
            w = w / max(w.sum(), 1e-20)
        weights[t], experts[t] = w * scale, e
        # exp(z - max) in fp32 is off by |z - max| U32 from its argument and a few
        # U32 of its own; the sum over E by the mean of that under the softmax,
        # ln E < 7, and its additions (E/64 + 6 < 22); topk additions, a division
        # and two products more.
        with np.errstate(invalid="ignore"):
            tol[t] = np.where(w > 0, (np.minimum(far[e], 200.0) + topk + 48) * U32 * w * scale, 0)
    return torch.from_numpy(weights), torch.from_numpy(experts), torch.from_numpy(tol)


def assert_route(got, want, what=""):
    weights, experts = (g.cpu() for g in got)
    w, e, tol = want
    assert weights.dtype == torch.float32 and experts.dtype == torch.int32
    assert torch.equal(experts, e), (what, (experts != e).nonzero()[:4].tolist(), experts[(experts != e).any(1)][:2],
                                     e[(experts != e).any(1)][:2])
    nan = w.isnan()
    assert torch.equal(weights.isnan(), nan), what
    err = (weights.double() - w).abs()[~nan]
    assert bool((err <= tol[~nan] + TINY["fp32"]).all()), (what, float((err - tol[~nan]).max()))


def dispatch(experts, E, x, x_scale=None, first=0):
    """(rows, row_scale, offsets, slots), rows and row_scale of offsets[E] rows."""
    ids = experts.long().numpy().astype(np.int64) - first
    T, topk = ids.shape
    flat = ids.reshape(-1)
    here = (flat >= 0) & (flat < E)
    order = np.argsort(np.where(here, flat, E), kind="stable")[:here.sum()]
    slots = np.full(T * topk, -1, np.int32)
    slots[order] = np.arange(len(order))
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat[here], minlength=E))]).astype(np.int32)
    token = torch.from_numpy(order // max(topk, 1))
    raw = x.contiguous().view(torch.uint8).reshape(x.shape[0], -1)[token] if x.numel() else None
    rows = raw.view(x.dtype).reshape(len(order), x.shape[1]) if raw is not None else x.new_zeros(len(order), x.shape[1])
    return (rows, None if x_scale is None else x_scale[token], torch.from_numpy(offsets),
            torch.from_numpy(slots.reshape(T, topk)))


def combine(rows, slots, weights, base=None):
    """(out, tol): topk fused multiply-adds in fp32, each off by U32 of a sum
    that stays below s = |base| + sum |weight * row|."""
    T, D = slots.shape[0], rows.shape[1]
    out = torch.zeros(T, D, dtype=torch.float64) if base is None else base.double().clone()
    s = out.abs()
    for j in range(slots.shape[1]):
        t = ((slots[:, j] >= 0) & (slots[:, j] < rows.shape[0])).nonzero()[:, 0]
        v = rows[slots[t, j].long()].double() * weights[t, j, None].double()
        out[t] += v
        s[t] += v.abs()
    return out, (slots.shape[1] + 2) * U32 * s


def adapters(y, x, A, B, ids, scales=None):
    """(out, tol, rms): out in 64 bits; tol, what no element may be off by in
    fp32: a sum of n products of 16-bit values is off by at most n U32 of the sum
    of their magnitudes, so the first product by K U32 and the second by R U32, and
    a few roundings more; rms, what the whole may be off by in the root mean square:
    independent roundings grow as the square root of their number, sqrt(K) U32 of
    a sum's size."""
    L, R, K = A.shape
    out, tol = y.double().clone(), torch.zeros(y.shape, dtype=torch.float64)
    delta = torch.zeros(y.shape, dtype=torch.float64)
    for a in range(L):
        t = (ids == a).nonzero()[:, 0]
        if not len(t):
            continue
        sc = 1.0 if scales is None else float(scales[a])
        xd, Ad, Bd = x[t].double(), A[a].double(), B[a].double()
        delta[t] = (xd @ Ad.t()) @ Bd.t() * sc
        tol[t] = (K + R + 64) * U32 * ((xd.abs() @ Ad.abs().t()) @ Bd.abs().t()) * abs(sc)
    out += delta
    tol += 2 * U32 * (y.double().abs() + delta.abs())
    rms = (K ** 0.5 + R ** 0.5 + 16) * U32 * float(delta.norm()) + 2 * U32 * float(y.double().norm())
    return out, tol, rms


def assert_close(got, ref, tol, out, what="", rms=None):
    got = got.cpu().double()
    assert got.shape == ref.shape
    err = (got - ref).abs()
    lim = tol + (ref.abs() + tol) * U_OUT[out] + TINY[out]
    assert bool((err <= lim).all()), (what, float((err - lim).max()), int((err > lim).sum()),
                                      (err > lim).nonzero()[:4].tolist())
    if rms is not None:
        assert float(err.norm()) <= rms + U_OUT[out] * float(ref.norm()) + TINY[out], (what, float(err.norm()), rms)
