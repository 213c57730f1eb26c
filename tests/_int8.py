"""Plain 64-bit forms of the int8 products, the token quantiser and the block
norm, on the CPU, and how far an fp32 evaluation may be from them.

U32 = 2^-24 is fp32's unit roundoff, U_OUT that of an output type (2^-p for p
significant bits: bf16 has 8, fp16 11, fp32 24; its half
step relative to the value; TINY its half subnormal step).
"""
import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
U32 = 2.0 ** -24
U_OUT = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11, "fp32": U32}
TINY = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}


def make_gemm(M, N, K, seed, bias=False, experts=None):
    r = np.random.default_rng(seed)
    d = {"A": r.integers(-128, 128, (M, K)).astype(np.int8),
         "a_s": r.uniform(0.001, 0.1, M).astype(np.float32)}
    shape = (N,) if experts is None else (experts, N)
    d["B"] = r.integers(-128, 128, (*shape, K)).astype(np.int8)
    d["b_s"] = r.uniform(0.0001, 0.01, shape).astype(np.float32)
    d["bias"] = r.standard_normal(N).astype(np.float32) if bias else None
    return {k: None if v is None else torch.from_numpy(v) for k, v in d.items()}


def sums(A, B):
    """The integer sums, exactly (below 2^53 in float64)."""
    return A.double() @ B.double().t()


def gemm_bits(d, out, acc=None):
    """The result with the roundings that the interface states: fl(fl(a_s *
    b_s) * fl(acc)), + bias, one rounding to the output type.  Bit for bit."""
    acc = sums(d["A"], d["B"]) if acc is None else acc
    c = (d["a_s"][:, None] * d["b_s"][None, :]) * acc.float()
    if d.get("bias") is not None:
        c = c + d["bias"]
    return c.to(DTYPES[out])


def assert_gemm(C, d, out, what=""):
    """Bit for bit against gemm_bits, and within the roundings' bound of the
    product in 64 bits: three relative errors of U32 on the product, one more
    on the sum with the bias, U_OUT for the output type."""
    got = C.cpu()
    want = gemm_bits(d, out)
    assert got.dtype == want.dtype and got.shape == want.shape
    bad = got != want
    assert not bool(bad.any()), (what, int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4], want[bad][:4])
    prod = sums(d["A"], d["B"]) * d["a_s"].double()[:, None] * d["b_s"].double()
    b = d["bias"].double() if d.get("bias") is not None else torch.zeros(1, dtype=torch.float64)
    ref = prod + b
    tol = ref.abs() * (U_OUT[out] * 1.01) + 5 * U32 * (prod.abs() + b.abs()) + TINY[out]
    over = (got.double() - ref).abs() > tol
    assert not bool((over & (ref.abs() < 65000)).any()), what


def quantize(x):
    """fp32 scales and codes by the stated rule (numpy's fp32 division is
    correctly rounded and rint rounds ties to even)."""
    v = x.float().numpy()
    with np.errstate(all="ignore"):
        amax = np.max(np.abs(v), axis=1, initial=0.0)
        s = (np.maximum(amax, np.float32(1e-12)) / np.float32(127)).astype(np.float32)
        t = (v / s[:, None]).astype(np.float32)
        q = np.rint(np.clip(np.where(np.isnan(t), np.float32(0), t), -127, 127))
    return torch.from_numpy(q.astype(np.int8)), torch.from_numpy(s)


def block_norm(h, x, post, gate, pre, alpha, eps, offset):
    """(r, y, tol_r, tol_y) in 64 bits.  A row sum of D squares has at most
    D/64 + 16 sequential fp32 additions in any of the kernels, so with
    c = D/64 + 24 roundings in all: |dr| <= c U32 s with
    s = |alpha x| + |gate u|; rms(r) is off by at most c U32 rms(s) from that
    and by c U32 relative from its own sum, so
    |dy| <= |pre| / rms (c U32 s) + |y| c U32 (1 + rms(s) / rms)."""
    h, D = h.double(), h.shape[1]
    c = (D / 64 + 24) * U32
    u = h
    if post is not None:
        u = h / torch.sqrt((h * h).mean(1, keepdim=True) + eps) * (post.double() + offset)
    if gate is not None:
        u = u * gate.double()
    ax = torch.zeros_like(h) if x is None else float(np.float32(alpha)) * x.double()
    r = ax + u
    s = ax.abs() + u.abs()
    tol_r = c * s
    if pre is None:
        return r, None, tol_r, None
    rms = torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    w = pre.double() + offset
    y = r / rms * w
    rms_s = torch.sqrt((s * s).mean(1, keepdim=True))
    tol_y = w.abs() / rms * tol_r + y.abs() * c * (1 + rms_s / rms)
    return r, y, tol_r, tol_y


def assert_close(got, ref, tol, out, what=""):
    got = got.cpu().double()
    lim = tol + ref.abs() * (U_OUT[out] * 1.01) + TINY[out]
    err = (got - ref).abs()
    assert bool((err <= lim).all()), (what, float((err - lim).max()), int((err > lim).sum()))


def assert_codes(q, scale, y, tol, fmt, what=""):
    """Codes and scales of y, known to within tol: the scale is the largest
    magnitude's (of the row, or of 128 columns) over the format's largest
    value, and code * scale is within half a step of y."""
    M, D = y.shape
    G, top = (1, 127.0) if fmt == "int8" else (D // 128, 448.0)
    yg, tg = y.view(M, G, -1), tol.view(M, G, -1)
    s = scale.cpu().double().view(M, G, 1)
    amax = yg.abs().amax(2, keepdim=True)
    want = amax.clamp(min=1e-12) / top
    assert bool(((s - want).abs() <= tg.amax(2, keepdim=True) / top + 2 * U32 * want).all()), what
    v = q.cpu().float().double().view(M, G, -1)
    if fmt == "int8":
        step = torch.ones_like(v)
    else:
        t = (yg / s).abs() + tg / s
        step = torch.exp2(torch.floor(torch.log2(t.clamp(min=2.0 ** -6))) - 3)
    err = (v * s - yg).abs()
    lim = 0.5 * step * s * (1 + 4 * U32) + tg + 4 * U32 * yg.abs()
    lim = torch.where(yg.abs() > top * s, (yg.abs() - top * s) + lim, lim)
    assert bool((err <= lim).all()), (what, float((err - lim).max()))
