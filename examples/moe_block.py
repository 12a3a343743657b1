"""A sparse (mixture-of-experts) SwiGLU block of a transformer, built from the
library's calls, for prompts and for single tokens.

    python examples/moe_block.py

Per block:  logits = H Wr               (router, swiglu_linear)
            route  = top-k experts, weights and expert order
            Y      = SiLU(H W1[e]) * (H W2[e]) for every routed row
            Z      = Y W3[e]
            R, H   = s R + g * RMSNorm(sum_j w_j Z_j),  RMSNorm of the new R

R is the residual stream, H the normalised input of the next block.  Group
sizes never leave the device, so the decode step is captured in a CUDA graph.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


class SparseBlock:
    """Weights of one block: `hidden` wide, `experts` SwiGLU experts of `inner` columns, `top_k` per token."""

    def __init__(self, hidden, inner, experts, top_k, *, seed=0, device="cuda", residual_scale=1.0, eps=1e-6):
        g = torch.Generator(device=device).manual_seed(seed)

        def weights(*shape, fan):
            return (torch.randn(*shape, generator=g, device=device) * fan**-0.5).bfloat16()
        self.Wr = weights(hidden, experts, fan=hidden)
        self.W1 = weights(experts, hidden, inner, fan=hidden)
        self.W2 = weights(experts, hidden, inner, fan=hidden)
        self.W3 = weights(experts, inner, hidden, fan=inner)
        self.post = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.pre = torch.ones(hidden, dtype=torch.bfloat16, device=device)
        self.gate = torch.full((hidden,), 0.5, dtype=torch.bfloat16, device=device)
        self.top_k, self.scale, self.eps = top_k, residual_scale, eps

    def __call__(self, R, H):
        import swiglu_gemm_transformer_gb300 as sg
        logits = sg.swiglu_linear(H, self.Wr)
        route = sg.swiglu_moe_route(logits, self.top_k, renormalize=True)
        Y = sg.swiglu_fused_grouped(H, self.W1, self.W2, route.offsets, route.rows)
        Z = sg.swiglu_linear_grouped(Y, self.W3, route.offsets)
        return sg.swiglu_residual_norm(Z, R, slots=route.slots, weights=route.weights, gamma_post=self.post,
                                       gate=self.gate, residual_scale=self.scale, gamma_pre=self.pre, eps=self.eps)

    def plain(self, R, H):
        """The same in elementary torch operations, 32 bits between the library's own roundings."""
        logits = (H.float() @ self.Wr.float()).bfloat16().float()
        top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
        ids, w = ids[:, :self.top_k], torch.softmax(top[:, :self.top_k], dim=1)
        x = H.float().unsqueeze(1).expand(-1, self.top_k, -1)
        out = torch.zeros_like(x)
        for e in range(self.W1.shape[0]):
            at = ids == e
            g, u = x[at] @ self.W1[e].float(), x[at] @ self.W2[e].float()
            y = (g / (1 + torch.exp(-g)) * u).bfloat16().float()
            out[at] = (y @ self.W3[e].float()).bfloat16().float()
        z = (w.unsqueeze(2) * out).sum(1)

        def norm(v):
            return v * torch.rsqrt((v * v).mean(1, keepdim=True) + self.eps)
        r = self.scale * R.float() + self.gate.float() * norm(z) * self.post.float()
        return r.to(R.dtype), (norm(r) * self.pre.float()).bfloat16()


class DecodeStep:
    """One token per sequence through `blocks`, captured once and replayed."""

    def __init__(self, blocks, batch, hidden, device="cuda"):
        self.R = torch.zeros(batch, hidden, device=device)
        self.H = torch.zeros(batch, hidden, dtype=torch.bfloat16, device=device)

        def step():
            R, H = self.R, self.H
            for b in blocks:
                R, H = b(R, H)
            return R, H
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            self.out = step()

    def __call__(self, R, H):
        self.R.copy_(R), self.H.copy_(H)
        self.graph.replay()
        return self.out


def main(hidden=512, inner=384, experts=16, top_k=4, layers=3, prompt=200):
    import swiglu_gemm_transformer_gb300 as sg
    blocks = [SparseBlock(hidden, inner, experts, top_k, seed=i) for i in range(layers)]
    g = torch.Generator(device="cuda").manual_seed(99)
    R = torch.randn(prompt, hidden, generator=g, device="cuda")
    H = (R * torch.rsqrt((R * R).mean(1, keepdim=True) + 1e-6)).bfloat16()
    # the prompt, block by block, against the plain form of each block
    worst = 0.0
    r, h = R, H
    for b in blocks:
        want = b.plain(r, h)
        r, h = b(r, h)
        worst = max(worst, float((r - want[0]).norm() / want[0].norm()))
    # single tokens: the prompt's rows one at a time give the prompt's results
    decode = DecodeStep(blocks, 1, hidden)
    off = max(float((decode(R[t:t + 1], H[t:t + 1])[0] - r[t:t + 1]).norm() / r[t:t + 1].norm()) for t in range(0, prompt, 40))
    rc, detail = sg.swiglu_device_status()
    if rc != sg.OK:
        raise RuntimeError(f"device status {sg.status_string(rc)} (detail {detail})")
    print(f"{layers} blocks, {prompt} tokens: off the plain form by {worst:.1e}; token by token off the prompt by {off:.1e}")
    return worst, off


if __name__ == "__main__":
    import __graft_entry__
    __graft_entry__.build()
    main()
