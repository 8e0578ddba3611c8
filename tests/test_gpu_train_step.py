"""The operators of a training step together: the example's stack against torch autograd in fp64, its
step against the oracle's, and a whole step as a captured graph."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import step_ops as so

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
D = torch.float64


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "moe_train", os.path.join(ROOT, "examples", "moe_train.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def logical(w1p, H, F):
    out = torch.empty(w1p.shape[0], H, 2 * F, dtype=w1p.dtype, device="cuda")
    g.moe_pack_fc1_weight(w1p, out, w1p.shape[0], H, F, 1, 64, 1)
    return out


def reference(stack, x, dh, H, F, scale):
    """The same stack in fp64 with autograd; the experts are those that the stack has chosen."""
    def norm(a):
        return a / torch.sqrt((a * a).mean(dim=1, keepdim=True) + 1e-6)

    leaf = {"x": x.to(D).requires_grad_()}
    for n, l in stack.names():
        t = getattr(stack, n)[l]
        leaf[n, l] = (logical(t, H, F) if n == "w1p" else t).to(D).requires_grad_()
    r = leaf["x"]
    h = norm(r) * leaf["w", 0]
    for l in range(stack.blocks):
        ids = stack.routers[l].topk_ids[:x.shape[0]].long()
        on = ids >= 0
        s = torch.sigmoid(h @ leaf["wr", l].t()).gather(1, ids.clamp(min=0)) * on
        w = scale * s / (s.sum(dim=1, keepdim=True) + 1e-20)
        o = torch.zeros_like(r)
        for e in range(leaf["w2", l].shape[0]):
            z = h @ leaf["w1p", l][e]
            out = (torch.nn.functional.silu(z[:, :F]) * z[:, F:]) @ leaf["w2", l][e]
            o = o + out * (w * (ids == e)).sum(dim=1, keepdim=True)
        r = r + norm(o) * leaf["wp", l + 1]
        h = norm(r) * leaf["w", l + 1]
    grads = torch.autograd.grad((h * dh.to(D)).sum(), list(leaf.values()))
    return h.detach(), dict(zip(leaf, grads))


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_stack_matches_autograd(lib, example):
    torch.manual_seed(0)
    T, H, F, scale = 300, 128, 192, 2.0
    stack = example.MoEStack(T, H, F, E=8, k=2, blocks=2, groups=4, of_groups=2, scale=scale)
    x, dh = torch.randn(T, H, device="cuda"), torch.randn(T, H, device="cuda").to(torch.bfloat16)
    mask = torch.rand(T, device="cuda") < 0.85
    h = stack.forward(x, mask).clone()
    dx = stack.backward(dh)
    want, grad = reference(stack, x, dh, H, F, scale)
    for b in range(2):
        ids = stack.routers[b].topk_ids[:T]
        assert (ids[~mask] == -1).all() and (ids[mask] >= 0).all()
        assert int(stack.counts[b].sum()) == 2 * int(mask.sum())
    # bf16 branches (2^-8 a rounding; half a dozen of them a block, two blocks)
    assert rel(h, want) <= 0.03 and rel(dx, grad["x"]) <= 0.03
    for (n, l), got in zip(stack.names(), stack.grads):
        got = logical(got, H, F) if n == "w1p" else got
        assert rel(got, grad[n, l]) <= 0.05, (n, l)


@pytest.mark.parametrize("bits", [8, 32])
def test_step_is_the_oracles(lib, example, bits):
    """The clipped AdamW step on the stack's own gradients."""
    T, H, F = 200, 128, 128
    stack = example.MoEStack(T, H, F, E=8, k=2, blocks=1, bits=bits, max_norm=1e-3)
    x = torch.randn(T, H, device="cuda")
    for t in (1, 2):
        stack.forward(x)
        stack.backward(torch.randn(T, H, device="cuda").to(torch.bfloat16))
        before = [(p if m is None else m).double().cpu().numpy().reshape(-1)
                  for p, m in zip(stack.params(), stack.opt.masters)]
        if bits == 32:
            old = [(m.double().cpu().numpy(), v.double().cpu().numpy())
                   for m, v in zip(stack.opt.m, stack.opt.v)]
        else:
            old = [(m.double().cpu().numpy(), v.double().cpu().numpy() ** 2)
                   for m, v in zip(*stack.opt.moments())]
        bias = stack.bias[0].clone()
        norm = float(stack.step())
        grads = [t_.double().cpu().numpy().reshape(-1) for t_ in stack.grads]
        want = math.sqrt(sum(float((v * v).sum()) for v in grads))
        assert abs(norm - want) <= 20 * 2.0 ** -24 * want and norm > 1e-3
        c = so.clip_factor(norm, 1e-3)
        for i, (n, _) in enumerate(stack.names()):
            decay = 0.1 if n in ("w1p", "w2") else 0.0
            p, _, _ = so.adamw(before[i], grads[i], *old[i], t, stack.lr, 0.9, 0.999, 1e-8, decay, c)
            master = stack.opt.masters[i]
            got = (stack.params()[i] if master is None else master).double().cpu().numpy().reshape(-1)
            # a move of at most some lr, 20 roundings of it and one of the weight (v starts at 0, its
            # root's error is relative)
            assert np.abs(got - p).max() <= 2.0 ** -24 * (2 * np.abs(p).max() + 400 * stack.lr)
        load = stack.counts[0].float()
        assert int(stack.opt.steps) == t and int(load.sum()) == T * 2  # every token's two experts
        moved = stack.bias[0] - bias
        assert torch.equal(torch.sign(moved), torch.sign(load.mean() - load))


def test_whole_step_in_a_graph(lib, example):
    """Forward, backward, clipping, AdamW and the bias's update captured once and replayed, against
    the same steps without a graph: bit for bit."""
    T, H, F = 256, 128, 128
    x = torch.randn(T, H, device="cuda")
    dh = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    ends = []
    for captured in (False, True):
        stack = example.MoEStack(T, H, F, E=8, k=2, blocks=2, bias_rate=0.01)

        def step():
            stack.forward(x)
            stack.backward(dh)
            stack.step()

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            again = graph.replay
        else:
            again = step
        for _ in range(3):
            again()
        torch.cuda.synchronize()
        assert int(stack.opt.steps) == 4
        ends.append([t.clone() for t in (*stack.params(), *stack.opt.m, *stack.opt.v, *stack.bias,
                                         stack.h[-1])])
    assert all(torch.equal(a, b) for a, b in zip(*ends))


def test_example_runs(lib, example, capsys):
    for bits in ("8", "32"):
        example.main(["--tokens", "256", "--hidden", "128", "--ffn", "128", "--steps", "2", "--bits",
                      bits])
    out = capsys.readouterr().out
    assert out.count("step ") == 4 and "nan" not in out
