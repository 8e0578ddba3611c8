"""One training step of a Mixture-of-Experts block on the library's kernels:

    h      = layer_norm(x)
    logits = h Wr^T                 router (a plain matrix product)
    y      = x + experts(h; top-k of logits) + shared_expert(h)
    loss   = <y, upstream> + balance loss of the router

and its backward pass down to x, with every weight gradient clipped by the global norm. The
routed experts run in BF16 (MoELayer), the shared expert's two projections in block-128 FP8
(Fp8Linear), its SwiGLU and the sums in torch.

    python examples/moe_block_step.py [--tokens 4096] [--hidden 1024] [--steps 3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import grouped_gemm_device_gb300 as g  # noqa: E402

BF16 = torch.bfloat16


class MoEBlock:
    """Weights, kernels' buffers and the step of one block."""

    def __init__(self, T, H, F, E=8, k=2, shared=None, coef=0.01, max_norm=1.0, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def weight(*shape, scale=0.02):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(BF16)

        S = F if shared is None else shared
        self.T, self.S, self.max_norm = T, S, max_norm
        self.gamma = torch.ones(H, dtype=BF16, device="cuda")
        self.beta = torch.zeros(H, dtype=BF16, device="cuda")
        self.wr = torch.randn(E, H, generator=gen, device="cuda") * 0.02  # router, fp32
        self.w1 = weight(E, H, 2 * F)                                     # [gate | linear]
        self.w1p, self.w2 = g.pack_w1(self.w1), weight(E, F, H)
        self.w_up, self.w_down = weight(2 * S, H), weight(H, S)
        self.norm = g.LayerNorm(H, T)
        self.router = g.RouterLoss(E, k, T, coef=coef)
        self.experts = g.MoELayer(g.make_desc(E=E, k=k, H=H, F=F, T_max=T))
        self.up, self.down = g.Fp8Linear(2 * S, H, T), g.Fp8Linear(H, S, T)
        self.clip = None

    def forward(self, x, token_mask=None):
        """x bf16 [T, H] -> (y bf16 [T, H], balance loss [1], per-expert counts [E])."""
        self.x, self.mask = x, token_mask
        h, _, _ = self.norm.forward(x, self.gamma, self.beta)
        self.h = h
        self.logits = h.float() @ self.wr.t()
        self.experts.route_permute(self.logits, h)
        aux, counts, _ = self.router.forward(self.logits, self.experts.topk_ids, token_mask)
        routed = self.experts.forward(self.w1p, self.w2, self.T)
        self.up.set_weight(self.w_up)      # the weights change every step
        self.down.set_weight(self.w_down)
        self.z = self.up.forward(h)
        gate, lin = self.z.float().split(self.S, dim=1)
        act = (torch.nn.functional.silu(gate) * lin).to(BF16)
        y = (x.float() + routed.float() + self.down.forward(act).float()).to(BF16)
        return y, aux, counts

    def backward(self, dy):
        """dy bf16 [T, H] -> dx bf16 [T, H]; leaves the clipped gradients in self.grads and the
        norm in self.grad_norm."""
        e = self.experts
        dh_routed, dw1p, dw2, d_probs = e.backward(dy, self.w1p, self.w2, self.T)
        d_logits = self.router.backward(self.logits, e.topk_ids, e.topk_probs, d_probs, self.mask)
        dh_router = d_logits @ self.wr
        dwr = d_logits.t() @ self.h.float()
        d_act, dw_down = self.down.backward(dy)
        gate, lin = self.z.float().split(self.S, dim=1)
        sig = torch.sigmoid(gate)
        d_gate = d_act.float() * lin * sig * (1 + gate * (1 - sig))
        d_lin = d_act.float() * gate * sig
        dh_shared, dw_up = self.up.backward(torch.cat([d_gate, d_lin], dim=1).to(BF16))
        dh = (dh_routed.float() + dh_router + dh_shared.float()).to(BF16)
        dx, dgamma, dbeta = self.norm.backward(dh, self.x, self.gamma)
        if self.clip is None:  # the gradients live in the layers' buffers: one plan for all steps
            self.dwr = torch.empty_like(dwr)
            self.grads = {"w1p": dw1p, "w2": dw2, "w_up": dw_up, "w_down": dw_down,
                          "wr": self.dwr, "gamma": dgamma, "beta": dbeta}
            self.clip = g.GradClip(self.grads.values())
        self.dwr.copy_(dwr)
        self.grad_norm = self.clip.clip(self.max_norm)
        return (dy.float() + dx.float()).to(BF16)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=8)
    ap.add_argument("--steps", type=int, default=3)
    a = ap.parse_args(argv)
    block = MoEBlock(a.tokens, a.hidden, a.ffn, a.experts)
    for step in range(a.steps):
        x = torch.randn(a.tokens, a.hidden, device="cuda").to(BF16)
        dy = (torch.randn(a.tokens, a.hidden, device="cuda") / a.tokens).to(BF16)
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        y, aux, counts = block.forward(x)
        dx = block.backward(dy)
        end.record()
        torch.cuda.synchronize()
        print(f"step {step}: {start.elapsed_time(end):.3f} ms  balance loss {float(aux):.5f}  "
              f"gradient norm {float(block.grad_norm):.4f}  tokens per expert {counts.tolist()}  "
              f"|y| {float(y.float().norm()):.1f}  |dx| {float(dx.float().norm()):.4f}")


if __name__ == "__main__":
    main()
