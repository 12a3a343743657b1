"""The sparse SwiGLU block of moe_block.py with 8-bit weights and a router by
scores: built from the library's calls, for prompts and for single tokens.

    python examples/moe_block_int8.py

Per block:  logits = H Wr                                 (router, swiglu_linear)
            route  = sigmoid scores with a bias for balance, the best groups'
                     top-k experts, renormalised weights
            Hq     = 8-bit codes of H by token
            Y      = SiLU(Hq W1[e]) * (Hq W2[e])          (8-bit weights by channel)
            Z      = Yq W3[e],  Yq = 8-bit codes of Y by row
            R, H   = s R + g * RMSNorm(sum_j w_j Z_j),  RMSNorm of the new R

The weights take half of the BF16 block's memory, which is what a few tokens'
time goes by.
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from examples.moe_block import DecodeStep, SparseBlock  # noqa: E402


class SparseBlockInt8(SparseBlock):
    """SparseBlock quantised: weights K-major, [experts, inner, hidden] and [experts, hidden, inner]."""

    def __init__(self, hidden, inner, experts, top_k, *, groups=4, kept_groups=2, seed=0, device="cuda", **kw):
        import swiglu_gemm_transformer_gb300 as sg
        super().__init__(hidden, inner, experts, top_k, seed=seed, device=device, **kw)
        g = torch.Generator(device=device).manual_seed(seed + 1000)
        self.bias = 0.05 * torch.randn(experts, generator=g, device=device)
        self.groups, self.kept = groups, kept_groups
        self.Q1, self.Q2, self.Q3 = (sg.swiglu_quant_int8(W.transpose(1, 2).contiguous()) for W in (self.W1, self.W2, self.W3))
        del self.W1, self.W2, self.W3

    def __call__(self, R, H, stages=None):
        """(R', H'); `stages`: a dict that gets what lies between."""
        import swiglu_gemm_transformer_gb300 as sg
        logits = sg.swiglu_linear(H, self.Wr)
        route = sg.swiglu_moe_route_scored(logits, self.top_k, bias=self.bias, groups=self.groups, kept_groups=self.kept)
        Hq = sg.swiglu_quant_int8(H)
        Y = sg.swiglu_fused_grouped_int8(*Hq, *self.Q1, *self.Q2, route.offsets, route.rows)
        Yq = sg.swiglu_quant_int8(Y)
        Z = sg.swiglu_linear_grouped_int8(*Yq, *self.Q3, route.offsets)
        out = sg.swiglu_residual_norm(Z, R, slots=route.slots, weights=route.weights, gamma_post=self.post, gate=self.gate,
                                      residual_scale=self.scale, gamma_pre=self.pre, eps=self.eps)
        if stages is not None:
            stages.update(logits=logits, route=route, Hq=Hq, Y=Y, Yq=Yq, Z=Z)
        return out

    def plain(self, R, H, logits=None):
        """The same in elementary torch operations, 32 bits between the library's own roundings; the router's
        choice may be taken from given logits (two roundings of one product can choose differently)."""
        E, k = self.Wr.shape[1], self.top_k
        if logits is None:
            logits = (H.float() @ self.Wr.float()).bfloat16()
        s = torch.sigmoid(logits.double())
        c = (s + self.bias.double()).view(-1, self.groups, E // self.groups)
        value = torch.sort(c, dim=2, descending=True).values[:, :, :2].sum(2)
        best = torch.sort(value, dim=1, descending=True, stable=True).indices[:, :self.kept]
        keep = torch.zeros_like(value, dtype=torch.bool).scatter_(1, best, True)
        c = torch.where(keep[:, :, None], c, -torch.inf).flatten(1)
        ids = torch.sort(c, dim=1, descending=True, stable=True).indices[:, :k]
        w = s.gather(1, ids)
        w = (w / w.sum(1, keepdim=True)).float()

        def codes(x):
            top = x.float().abs().amax(-1, keepdim=True)
            q = torch.round(127 * x.double() / top.double()).float()
            return torch.where(top > 0, q, 0.0), top / 127

        def product(x, e, Q):
            q, sx = codes(x)
            return (q @ Q[0][e].float().t()) * sx * Q[1][e]
        x = H.unsqueeze(1).expand(-1, k, -1)
        out = torch.zeros(x.shape, device=H.device)
        for e in range(E):
            at = ids == e
            g, u = product(x[at], e, self.Q1), product(x[at], e, self.Q2)
            out[at] = product((g / (1 + torch.exp(-g)) * u).bfloat16(), e, self.Q3).bfloat16().float()
        z = (w.unsqueeze(2) * out).sum(1)

        def norm(v):
            return v * torch.rsqrt((v * v).mean(1, keepdim=True) + self.eps)
        r = self.scale * R.float() + self.gate.float() * norm(z) * self.post.float()
        return r.to(R.dtype), (norm(r) * self.pre.float()).bfloat16()


def main(hidden=512, inner=384, experts=16, top_k=4, layers=3, prompt=200):
    import swiglu_gemm_transformer_gb300 as sg
    blocks = [SparseBlockInt8(hidden, inner, experts, top_k, seed=i) for i in range(layers)]
    g = torch.Generator(device="cuda").manual_seed(99)
    R = torch.randn(prompt, hidden, generator=g, device="cuda")
    H = (R * torch.rsqrt((R * R).mean(1, keepdim=True) + 1e-6)).bfloat16()
    # the prompt, block by block, against the plain form of each block
    worst = 0.0
    r, h = R, H
    for b in blocks:
        stages = {}
        got = b(r, h, stages)
        want = b.plain(r, h, stages["logits"])
        r, h = got
        worst = max(worst, float((r - want[0]).norm() / want[0].norm()))
    # single tokens, one at a time, through one captured step
    decode = DecodeStep(blocks[:1], 1, hidden)
    first = blocks[0](R, H)[0]
    off = max(float((decode(R[t:t + 1], H[t:t + 1])[0] - first[t:t + 1]).norm() / first[t:t + 1].norm()) for t in range(0, prompt, 40))
    rc, detail = sg.swiglu_device_status()
    if rc != sg.OK:
        raise RuntimeError(f"device status {sg.status_string(rc)} (detail {detail})")
    print(f"{layers} blocks, {prompt} tokens: off the plain form by {worst:.1e}; token by token off the prompt by {off:.1e}")
    return worst, off


if __name__ == "__main__":
    import __graft_entry__
    __graft_entry__.build()
    main()
