"""Training steps of a stack of Mixture-of-Experts blocks on the library's kernels:

    h_0 = w_0 N(x_0);   o_l = experts(h_l) under a routing with groups and a balance bias
    x_{l+1} = x_l + wp_{l+1} N(o_l),   h_{l+1} = w_{l+1} N(x_{l+1})        loss = <h_L, target>

on an fp32 residual stream, with bf16 expert weights, their fp32 masters in AdamW (states in 8 or 32
bits) and gradients clipped within the optimiser's step. The bias of an expert moves against its load.

    python examples/moe_train.py [--tokens 4096] [--hidden 1024] [--blocks 2] [--steps 3] [--bits 8]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
import grouped_gemm_device_gb300 as g  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


class MoEStack:
    """Weights, kernels' buffers and the step of `blocks` blocks for up to T tokens."""

    def __init__(self, T, H, F, E=16, k=4, blocks=2, groups=4, of_groups=2, scale=2.0, bits=8,
                 lr=1e-3, max_norm=1.0, bias_rate=1e-3, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def weight(*shape, dtype=BF16, scale=0.02):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

        self.blocks, self.max_norm, self.bias_rate = blocks, max_norm, bias_rate
        self.w = [torch.ones(H, device="cuda") for _ in range(blocks + 1)]
        self.wp = [None] + [torch.full((H,), 0.5, device="cuda") for _ in range(blocks)]
        self.wr = [weight(E, H, dtype=F32, scale=1 / math.sqrt(H)) for _ in range(blocks)]
        self.w1p = [g.pack_w1(weight(E, H, 2 * F, scale=1 / math.sqrt(H))) for _ in range(blocks)]
        self.w2 = [weight(E, F, H, scale=1 / math.sqrt(F)) for _ in range(blocks)]
        self.bias = [torch.zeros(E, device="cuda") for _ in range(blocks)]
        self.norms = [g.ResidualNorm(H, T, dtype=F32, branch_dtype=BF16, weight_dtype=F32,
                                     post_norm=True) for _ in range(blocks + 1)]
        self.routers = [g.RouterTopK(E, k, T, score="sigmoid", n_group=groups,
                                     topk_group=of_groups, group_top=2, scale=scale)
                        for _ in range(blocks)]
        desc = g.make_desc(E=E, k=k, H=H, F=F, T_max=T)
        self.experts = [g.MoELayer(desc) for _ in range(blocks)]
        self.lr, self.bits, self.opt = lr, bits, None

    def forward(self, x, mask=None):
        """x fp32 [T, H], mask bool [T] (False: padding, which no expert sees) -> h bf16 [T, H]."""
        T = x.shape[0]
        x, h = self.norms[0].forward(x, weight=self.w[0])
        self.x, self.h, self.o, self.logits, self.counts = [x], [h], [None], [], []
        for l in range(self.blocks):
            logits = self.h[l].float() @ self.wr[l].t()
            ids, weights, counts = self.routers[l].forward(logits, self.bias[l], mask)
            self.experts[l].permute(ids, weights, self.h[l])
            o = self.experts[l].forward(self.w1p[l], self.w2[l], T)
            x, h = self.norms[l + 1].forward(self.x[l], o, self.w[l + 1], self.wp[l + 1])
            self.x.append(x)
            self.h.append(h)
            self.o.append(o)
            self.logits.append(logits)
            self.counts.append(counts)
        return h

    def backward(self, dh):
        """dh bf16 [T, H] -> dx fp32 [T, H]; leaves the weights' gradients in self.grads, in the order
        of self.params()."""
        T, dx = dh.shape[0], None
        d = {}
        for l in range(self.blocks, -1, -1):
            dx, do, d["w", l], d["wp", l], _ = self.norms[l].backward(
                dh, self.x[l], self.o[l], self.w[l], self.wp[l], dx_new=dx)
            if l == 0:
                break
            b = l - 1
            dh_experts, d["w1p", b], d["w2", b], d_weights = self.experts[b].backward(
                do, self.w1p[b], self.w2[b], T)
            d_logits = self.routers[b].backward(self.logits[b], d_weights)
            d["wr", b] = d_logits.t() @ self.h[b].float()
            dh = (dh_experts.float() + d_logits @ self.wr[b]).to(BF16)
        grads = [d[name] for name in self.names()]
        if self.opt is None:  # most gradients live in the kernels' buffers: one plan for all steps
            self.grads = [t if key[0] != "wr" else torch.empty_like(t)
                          for key, t in zip(self.names(), grads)]
            decay = [0.1 if key[0] in ("w1p", "w2") else 0.0 for key in self.names()]
            self.clip = g.GradClip(self.grads)
            self.opt = g.AdamW(self.params(), self.grads, lr=self.lr, weight_decay=decay,
                               state_bits=self.bits)
        for key, mine, t in zip(self.names(), self.grads, grads):
            if key[0] == "wr":
                mine.copy_(t)
        return dx

    def names(self):
        return ([("w", l) for l in range(self.blocks + 1)]
                + [("wp", l) for l in range(1, self.blocks + 1)]
                + [(n, l) for l in range(self.blocks) for n in ("wr", "w1p", "w2")])

    def params(self):
        return [getattr(self, n)[l] for n, l in self.names()]

    def step(self):
        """The optimiser's step on the last backward's gradients; returns their norm [1]."""
        norm = self.clip.clip(math.inf)
        self.opt.step(norm=norm, max_norm=self.max_norm)
        for bias, counts in zip(self.bias, self.counts):
            load = counts.float()
            bias += self.bias_rate * torch.sign(load.mean() - load)
        return norm


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--ffn", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args(argv)
    stack = MoEStack(a.tokens, a.hidden, a.ffn, a.experts, blocks=a.blocks, bits=a.bits)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    x = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda")
    dh = torch.randn(a.tokens, a.hidden, generator=gen, device="cuda") / a.tokens
    for step in range(a.steps):
        start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        start.record()
        h = stack.forward(x)
        loss = (h.float() * dh).sum()
        stack.backward(dh.to(BF16))
        norm = stack.step()
        end.record()
        torch.cuda.synchronize()
        print(f"step {step}: {start.elapsed_time(end):.3f} ms  loss {float(loss):.5f}  gradient "
              f"norm {float(norm):.4f}  tokens per expert {stack.counts[-1].tolist()}")


if __name__ == "__main__":
    main()
