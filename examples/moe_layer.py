"""One MoE layer around the load balancer: the router's choice, the counted and
redirected ids, rows grouped by physical slot, the experts' products in 8-bit
blocks, in 16 bits or with 4-bit weights, and the weighted sum; then training
steps of it with the balance loss, in 8-bit blocks or 16 bits.  Run on an MI355X:

    python examples/moe_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_load_eplb_amd as eplb
from moe_expert_load_eplb_amd.autograd import combine, expert_linear, expert_linear16, route


class MoELayer:
    """E logical experts of two matrices (C -> 2 F, gated, F -> C), held as P
    physical replicas placed on RK ranks of N nodes; all on this GPU.  bits: of
    the products, 8 (both operands), 16 (both) or 4 (the weights; 16 in training)."""

    def __init__(self, C=256, F=128, E=32, K=4, P=40, G=4, N=2, RK=4, window=8, device="cuda", seed=0, bits=8):
        g = torch.Generator(device=device).manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g, device=device) * shape[-1] ** -0.5).bfloat16()

        self.C, self.F, self.E, self.K, self.P, self.G, self.N, self.RK, self.bits = C, F, E, K, P, G, N, RK, bits
        self.router, self.up, self.down = weight(E, C).float(), weight(E, 2 * F, C), weight(E, C, F)
        self.bias = torch.zeros((E,), device=device)
        self.ring = torch.zeros((window, 1, E), dtype=torch.int32, device=device)
        self.step = 0
        self.place(torch.ones((1, E), dtype=torch.int64, device=device))

    def place(self, load):
        """A new placement from the loads, and the replicas' weights laid out for it."""
        self.phy2log, self.log2phy, self.logcnt, status = eplb.rebalance(load, self.P, self.G, self.N, self.RK)
        held = self.phy2log[0].long()
        held_as = {8: eplb.quantize_weights, 16: lambda w: (w,), 4: eplb.quantize_weights4}[self.bits]
        self.up_held, self.down_held = held_as(self.up[held]), held_as(self.down[held])

    def product(self, x, w, offsets, rows=None, K=1):
        if self.bits == 8:
            return eplb.expert_matmul(*eplb.quantize_rows(x), *w, offsets, rows=rows, K=K)
        return (eplb.expert_matmul16 if self.bits == 16 else eplb.expert_matmul4)(x, *w, offsets, rows=rows, K=K)

    def logits(self, x):
        return x.float() @ self.router.t()

    def serve(self, x):
        """x [T, C] bfloat16 -> [T, C]; counts the step's load into the window."""
        T, K = x.shape[0], self.K
        ids, weights = eplb.gate(self.logits(x), K, bias=self.bias, G=self.G, top_groups=self.G // 2, group_top=2)
        self.load, _, slots = eplb.hist_redirect(ids.view(1, T, K), self.E, self.ring, self.step, self.log2phy,
                                                 self.logcnt)
        self.step += 1
        offsets, order, place = (t[0] for t in eplb.group_rows(slots, self.P))
        h = self.product(x, self.up_held, offsets, order, K)
        a, b = h.float().chunk(2, dim=1)
        h = (torch.nn.functional.silu(a) * b).bfloat16()
        return eplb.combine_rows(self.product(h, self.down_held, offsets), place, weights)

    def train(self, x, seg, alpha=0.01):
        """x [T, C] bfloat16, seg [S + 1]: (output [T, C], balance loss [S]), differentiable in x, router, up and down."""
        T, K = x.shape[0], self.K
        ids, weights, loss, counts, prob, tokens = route(self.logits(x), K, seg, alpha, bias=self.bias, G=self.G,
                                                         top_groups=self.G // 2, group_top=2)
        offsets, order, place = (t[0] for t in eplb.group_rows(ids.view(1, T, K), self.E))
        linear = expert_linear if self.bits == 8 else expert_linear16
        h = linear(x, self.up, offsets, order, place, K)
        a, b = h.float().chunk(2, dim=1)
        y = linear((torch.nn.functional.silu(a) * b).bfloat16(), self.down, offsets)
        return combine(y, weights, place, order, dtype=torch.float32), loss


def main():
    layer = MoELayer()
    g = torch.Generator(device="cuda").manual_seed(1)
    for step in range(16):
        x = torch.randn((64, layer.C), generator=g, device="cuda").bfloat16()
        y = layer.serve(x)
        if step % 8 == 7:
            layer.place(layer.load)
    print(f"served 16 steps of 64 tokens, output norm {y.float().norm():.3f}, replicas {layer.logcnt[0].tolist()}")
    x = torch.randn((64, layer.C), generator=g, device="cuda").bfloat16()
    for bits in (16, 4):
        y = MoELayer(bits=bits).serve(x)
        print(f"the products in {bits} bits: 64 tokens, output norm {y.float().norm():.3f}")
    seg = torch.tensor([0, 100, 256], dtype=torch.int32, device="cuda")
    x = torch.randn((256, layer.C), generator=g, device="cuda").bfloat16()
    target = torch.randn((256, layer.C), generator=g, device="cuda") * 0.1
    params = [layer.router, layer.up, layer.down]
    for p in params:
        p.requires_grad_(True)
    for step in range(5):
        out, balance = layer.train(x, seg)
        loss = ((out - target) ** 2).mean() + balance.mean()
        grads = torch.autograd.grad(loss, params)
        with torch.no_grad():
            for p, d in zip(params, grads):
                p -= (0.5 * d.float() / d.float().norm()).to(p.dtype)
        print(f"step {step}: loss {loss.item():.4f}, balance {balance.tolist()}")


if __name__ == "__main__":
    main()
