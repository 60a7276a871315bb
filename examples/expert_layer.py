"""A MoE layer whose expert matrices are the caller's own, in bf16 or in microscaled 4-bit floating point (MXFP4):

    router (moe_route) -> (token, expert) pairs sorted by expert -> gate/up product of each expert's rows -> SwiGLU
    -> down product -> the rows back to their tokens, weighted, on top of the shared expert's

Run it on a GPU with `python examples/expert_layer.py [tokens]`: it prints each kernel's GPU time and how far the outputs
are from the same layer computed in float64 from the same weights.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gen import inputs as gen  # noqa: E402
from int4_routed_expert_amd import moe as M  # noqa: E402

BF = torch.bfloat16


class Layer:
    """Seeded weights of the tiny configuration's routing and sizes; `mx` holds them in 4 bits, quantised when loaded."""

    def __init__(self, mx: bool, seed=0):
        w = gen.WORKLOADS["tiny"]
        c = self.c = w.cfg
        self.mx, self.cfg = mx, M.make_cfg(c)
        self.router, self.bias = torch.from_numpy(gen.router_weights(w)).cuda(), torch.from_numpy(gen.router_bias(w)).cuda()
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            return (torch.randn(*shape, generator=g, device="cuda") / math.sqrt(shape[-1])).to(BF)

        E, H, I, Is = c.n_experts, c.hidden, c.moe_inter, c.shared_inter
        self.plain = {"gate_up": weight(E, 2 * I, H), "down": weight(E, H, I),
                      "shared_gate_up": weight(1, 2 * Is, H), "shared_down": weight(1, H, Is)}
        self.packed = {}
        for name, m in self.plain.items() if mx else ():
            q, e = M.mx_quant(m.flatten(0, 1))
            self.packed[name] = q.view(*m.shape[:2], -1), e.view(*m.shape[:2], -1)

    def forward(self, x):
        """y [S, H] fp32 of the rows x [S, H] bf16."""
        c, k = self.c, self.c.top_k
        idx, weights = M.route(x, self.router, self.bias, self.cfg)
        first, order, place = M.group(idx, c.n_experts)
        if self.mx:
            p = self.packed
            rows = M.mx_quant(x)
            act = M.mx_silu_quant(M.mx_grouped_matmul(*rows, *p["gate_up"], first, order, k))
            z = M.mx_grouped_matmul(*act, *p["down"], first)
            act = M.mx_silu_quant(M.mx_matmul(*rows, *(t[0] for t in p["shared_gate_up"])))
            shared = M.mx_matmul(*act, *(t[0] for t in p["shared_down"]))
        else:
            p = self.plain
            gate_up = M.grouped_matmul(x, p["gate_up"], first, order, k)
            z = M.grouped_matmul(M.silu_quant(gate_up, y_dtype=BF, quant=False)[0], p["down"], first)
            every = torch.arange(2, dtype=torch.int32, device=x.device) * len(x)  # the shared expert has all rows
            gate_up = M.grouped_matmul(x, p["shared_gate_up"], every)
            shared = M.grouped_matmul(M.silu_quant(gate_up, y_dtype=BF, quant=False)[0], p["shared_down"], every)
        return M.combine(z, weights, place, add=shared, out_dtype=torch.float32)


def reference(layer, x):
    """The layer in float64 from the weights as it holds them, activations not rounded at all."""
    c = layer.c
    w = {name: (M.mx_values(*(t.flatten(0, 1) for t in layer.packed[name]), dtype=torch.float32).view(m.shape) if layer.mx else m).double()
         for name, m in layer.plain.items()}

    def ffn(v, gate_up, down):
        g, u = (v @ gate_up.t().contiguous()).chunk(2, 1)
        return (g * torch.sigmoid(g) * u) @ down.t().contiguous()

    idx, weights = M.route(x, layer.router, layer.bias, layer.cfg)
    v = x.double()
    y = ffn(v, w["shared_gate_up"][0], w["shared_down"][0])
    for e in range(c.n_experts):
        tokens, choice = (idx == e).nonzero(as_tuple=True)
        if len(tokens):
            y[tokens] += weights[tokens, choice].double()[:, None] * ffn(v[tokens], w["gate_up"][e], w["down"][e])
    return y


def main():
    S = int(sys.argv[1]) if len(sys.argv) > 1 else 16
    for mx in (False, True):
        layer = Layer(mx)
        x = torch.randn(S, layer.c.hidden, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF)
        layer.forward(x)
        M.moe_profile_enable(True)
        y = layer.forward(x)
        times = M.moe_profile_report()
        M.moe_profile_enable(False)
        print("experts in MXFP4" if mx else "experts in bf16")
        for name, (ms, n) in times.items():
            print(f"  {name:22s} {n} x {ms / n * 1e3:7.2f} us")
        want = reference(layer, x)
        print(f"  {((y.double() - want).norm() / want.norm()).item():.2e} from float64")


if __name__ == "__main__":
    main()
