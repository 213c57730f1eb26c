"""One mixture-of-experts block in 8-bit integers, as a decoder runs it between
two attention blocks:

    r, q, s = block_norm(attention output, residual, .., quantize="int8")
    router on r, tokens sorted by expert
    up   = int8_grouped_gemm(q of the sorted tokens, ..)      [2F per expert]
    act  = silu(up[:, :F]) * up[:, F:]                         -> quantize_tokens
    down = int8_grouped_gemm(act, ..)                          [D per expert]
    h    = sum of each token's experts, weighted by the router
    r, q, s = block_norm(h, r, .., quantize="int8")
    qkv  = int8_gemm(q, s, next projection)

Nothing here waits for the GPU: the experts' row counts stay on it.

    python3 examples/int8_moe_block.py [--tokens 64]

prints the block's relative error against the same block in 64-bit floating
point on the unquantised weights, and its time per call.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_fp8_gemm_amd as fbg  # noqa: E402


class Int8MoEBlock:
    def __init__(self, D=1024, F=512, E=32, topk=4, out=1536, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device=device)
        self.E, self.topk, self.F = E, topk, F
        self.router = rn(E, D) / D ** 0.5
        self.w_up, self.w_down = rn(E, 2 * F, D) / D ** 0.5, rn(E, D, F) / F ** 0.5
        self.w_next = rn(out, D) / D ** 0.5
        bf = lambda t: t.to(torch.bfloat16)
        self.norms = [bf(1 + 0.1 * rn(D)) for _ in range(4)]    # after and before, for both boundaries
        self.gates = [bf(torch.sigmoid(rn(D))) for _ in range(2)]
        self.scale = 0.875
        # Weights once: int8 codes and one scale per output channel.
        up, up_s = fbg.quantize_tokens(self.w_up.view(E * 2 * F, D))
        down, down_s = fbg.quantize_tokens(self.w_down.view(E * D, F))
        self.up, self.up_s = up.view(E, 2 * F, D), up_s.view(E, 2 * F)
        self.down, self.down_s = down.view(E, D, F), down_s.view(E, D)
        self.next, self.next_s = fbg.quantize_tokens(self.w_next)

    def route(self, r):
        """Weights [T, topk], and each token's experts."""
        weight, expert = torch.topk(torch.softmax(r.float() @ self.router.t(), dim=-1), self.topk, dim=-1)
        return weight / weight.sum(dim=-1, keepdim=True), expert

    def __call__(self, attention, residual):
        T, D = attention.shape
        r, q, s = fbg.block_norm(attention, residual, post_weight=self.norms[0], gate=self.gates[0],
                                 pre_weight=self.norms[1], residual_scale=self.scale, quantize="int8")
        weight, expert = self.route(r)
        order = torch.argsort(expert.reshape(-1), stable=True)
        token = order // self.topk
        # offsets[e]: rows whose expert is below e (no atomics, no wait for the GPU)
        ids = torch.arange(self.E + 1, device=q.device)
        offsets = torch.searchsorted(expert.reshape(-1)[order], ids).to(torch.int32)
        up = fbg.int8_grouped_gemm(q[token], s[token], self.up, self.up_s, offsets)
        act = torch.nn.functional.silu(up[:, :self.F]) * up[:, self.F:]
        down = fbg.int8_grouped_gemm(*fbg.quantize_tokens(act), self.down, self.down_s, offsets, out_dtype=torch.float32)
        # back to token order: row order[i] of the (token, choice) matrix is row i here
        rows = torch.empty_like(down)
        rows[order] = down
        h = (rows.view(T, self.topk, D) * weight[..., None]).sum(dim=1).to(torch.bfloat16)
        r, q, s = fbg.block_norm(h, r, post_weight=self.norms[2], gate=self.gates[1], pre_weight=self.norms[3],
                                 residual_scale=self.scale, quantize="int8")
        return r, fbg.int8_gemm(q, s, self.next, self.next_s), expert

    def reference(self, attention, residual, expert):
        """The same block in 64 bits on the unquantised weights, for the experts
        that the router picked."""
        rms = lambda v, w: v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + 1e-6) * w.double()
        r = self.scale * residual.double() + self.gates[0].double() * rms(attention.double(), self.norms[0])
        y = rms(r, self.norms[1])
        p = torch.softmax(r @ self.router.double().t(), dim=-1).gather(1, expert)
        p = p / p.sum(dim=-1, keepdim=True)
        h = torch.zeros_like(r)
        for e in range(self.E):
            t, c = (expert == e).nonzero(as_tuple=True)
            if len(t):
                up = y[t] @ self.w_up[e].double().t().contiguous()
                act = torch.nn.functional.silu(up[:, :self.F]) * up[:, self.F:]
                h.index_add_(0, t, (act @ self.w_down[e].double().t().contiguous()) * p[t, c][:, None])
        r = self.scale * r + self.gates[1].double() * rms(h, self.norms[2])
        return r, rms(r, self.norms[3]) @ self.w_next.double().t().contiguous()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=64)
    a = ap.parse_args()
    block = Int8MoEBlock()
    g = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.randn(a.tokens, 1024, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    r, out, expert = block(x, res)
    want_r, want = block.reference(x, res, expert)
    off = lambda u, v: float((u.double() - v).norm() / v.norm())
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        block(x, res)
    start.record()
    for _ in range(20):
        block(x, res)
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens: relative error of the residual {off(r, want_r):.2e}, of the next projection "
          f"{off(out, want):.2e}; {start.elapsed_time(end) / 20 * 1e3:.0f} us a call")


if __name__ == "__main__":
    main()
