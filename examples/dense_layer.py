"""A decoder layer's dense path around its MoE layer, in int8 (W8A8), for one call of S tokens:

    residual sum and norm -> q/k/v product -> rotary positions -> attention (the caller's own; a plain one stands in here)
    -> residual sum and norm -> gate/up product -> SwiGLU -> down product      (a dense layer's FFN)
    -> residual sum and norm -> router and routed experts (moe_layer)          (the MoE layer after it)

Run it on a GPU with `python examples/dense_layer.py [tokens]`: it prints each call's GPU time and how far the outputs
are from the same layer computed in float64 from the same int8 weights.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gen import inputs as gen  # noqa: E402
from int4_routed_expert_amd import moe as M  # noqa: E402

EPS = 1e-5
HEADS, KHEADS, D, ROT = 8, 2, 64, 32  # the last ROT of a head's D dimensions turn


def quantise_weights(w):
    """(int8 [N, K], fp32 [N]): a weight matrix as MOE_WF_Q8_ROW holds it, once, when a model is loaded."""
    scale = w.abs().amax(1) / 127
    return (w / scale[:, None]).round().to(torch.int8), scale


class Layer:
    """Seeded weights of a dense layer of the tiny configuration's width and of the MoE layer that follows it."""

    def __init__(self, inter=768, seed=0):
        w = gen.WORKLOADS["tiny"]
        c = self.c = w.cfg
        H = c.hidden
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(n, k):
            return quantise_weights(torch.randn(n, k, generator=g, device="cuda") / math.sqrt(k))

        self.gammas = [(1 + 0.1 * torch.randn(H, generator=g, device="cuda")).bfloat16() for _ in range(3)]
        self.qkv = weight((HEADS + 2 * KHEADS) * D, H)
        self.out = (torch.randn(H, HEADS * D, generator=g, device="cuda") / math.sqrt(HEADS * D)).bfloat16()
        self.gate_up = weight(2 * inter, H)
        self.down = weight(H, inter)
        self.freqs, self.factor = M.rope_freqs(ROT, 10000.0, "yarn", 4.0, 4096)
        # the MoE layer: router, packed experts in their slots, shared expert
        self.cfg = M.make_cfg(c)
        size = M.moe_expert_bytes(self.cfg, c.moe_inter)
        self.slab = torch.empty(c.n_experts * size, dtype=torch.uint8, device="cuda")
        self.shared = torch.empty(M.moe_expert_bytes(self.cfg, c.shared_inter), dtype=torch.uint8, device="cuda")
        for e in range(c.n_experts + 1):
            x = gen.expert_weights(w, 0, e)
            to = self.slab[e * size:(e + 1) * size] if e < c.n_experts else self.shared
            M.pack_expert(self.cfg, x.inter, *[torch.from_numpy(a).cuda() for a in x.parts()], to, 1)
        self.view = M.slot_view(self.slab, size, torch.arange(c.n_experts, dtype=torch.int32, device="cuda"), c.n_experts)
        self.router = torch.from_numpy(gen.router_weights(w)).cuda()
        self.bias = torch.from_numpy(gen.router_bias(w)).cuda()

    def forward(self, h, x, pos):
        """(h, x, y): the residual stream h [S, H] with x, the previous layer's output, added; then the dense layer's and
        the MoE layer's outputs added to it in turn.  h and x are bf16; h is updated in place."""
        S = h.shape[0]
        h, _, q, d = M.norm_quant(x, self.gammas[0], EPS, residual=h, h=h)
        qkv = M.qmatmul(q, d, *self.qkv).view(S, HEADS + 2 * KHEADS, D)
        q, k, v = qkv.split((HEADS, KHEADS, KHEADS), 1)
        q, k = M.rope(q, k, pos, self.freqs, offset=D - ROT, interleaved=True, factor=self.factor, inplace=True)
        x = (attention(q, k, v) @ self.out.t().float()).bfloat16()
        h, _, q, d = M.norm_quant(x, self.gammas[1], EPS, residual=h, h=h)
        _, q, d = M.silu_quant(M.qmatmul(q, d, *self.gate_up))
        x = M.qmatmul(q, d, *self.down)
        h, y, _, _ = M.norm_quant(x, self.gammas[2], EPS, residual=h, h=h, y_dtype=torch.bfloat16, quant=False)
        _, _, moe = M.layer(y, self.router, self.bias, self.view, self.shared, self.cfg)
        return h, y, moe


def attention(q, k, v):
    """Causal attention with grouped keys, plain: what a caller brings along.  [S, heads * D] fp32."""
    S = q.shape[0]
    q, k, v = (t.float().transpose(0, 1).contiguous() for t in (q, k, v))
    k, v = (t.repeat_interleave(HEADS // KHEADS, 0) for t in (k, v))
    score = torch.bmm(q, k.transpose(1, 2).contiguous()) / math.sqrt(D)
    score = score.masked_fill(torch.ones(S, S, dtype=torch.bool, device=q.device).triu(1), -math.inf)
    return torch.bmm(score.softmax(-1), v).transpose(0, 1).reshape(S, HEADS * D)


def reference(layer, h, x, pos):
    """The dense part in float64 from the same weights: int8 weights, activations not rounded at all."""
    def norm(v, gamma):
        return v * torch.rsqrt(v.square().mean(1, keepdim=True) + EPS) * gamma.double()

    def product(v, w):
        return v @ (w[0].double() * w[1].double()[:, None]).t()

    S = h.shape[0]
    h = h.double() + x.double()
    qkv = product(norm(h, layer.gammas[0]), layer.qkv).view(S, -1, D)
    a = pos.double()[:, None, None] * layer.freqs
    c, s = a.cos() * layer.factor, a.sin() * layer.factor
    turned = qkv.clone()
    even, odd = qkv[..., D - ROT::2], qkv[..., D - ROT + 1::2]
    turned[..., D - ROT::2], turned[..., D - ROT + 1::2] = even * c - odd * s, odd * c + even * s
    q, k, v = turned[:, :HEADS], turned[:, HEADS:HEADS + KHEADS], qkv[:, HEADS + KHEADS:]
    h = h + attention(q, k, v).double() @ layer.out.t().double()
    g, u = product(norm(h, layer.gammas[1]), layer.gate_up).chunk(2, 1)
    h = h + product(g * torch.sigmoid(g) * u, layer.down)
    return h, norm(h, layer.gammas[2])


def inputs(layer, S, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    h, x = (torch.randn(S, layer.c.hidden, generator=g, device="cuda").bfloat16() for _ in range(2))
    return h, x, torch.arange(S, device="cuda") + 5000


def main():
    S = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    layer = Layer()
    h, x, pos = inputs(layer, S)
    want_h, want_y = reference(layer, h, x, pos)
    layer.forward(h.clone(), x, pos)
    M.moe_profile_enable(True)
    got_h, got_y, moe = layer.forward(h.clone(), x, pos)
    times = M.moe_profile_report()
    M.moe_profile_enable(False)
    for name, (ms, n) in times.items():
        print(f"{name:22s} {n} x {ms / n * 1e3:7.2f} us")
    for name, got, want in (("residual stream", got_h, want_h), ("MoE layer's input", got_y, want_y)):
        print(f"{name}: {((got.double() - want).norm() / want.norm()).item():.2e} from float64 (activations in int8 and bf16)")
    print(f"MoE layer's output: {tuple(moe.shape)} {moe.dtype}, finite: {bool(torch.isfinite(moe).all())}")


if __name__ == "__main__":
    main()
