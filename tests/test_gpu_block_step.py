"""The example's training step of a block against torch autograd in fp64 on unquantised values."""
import importlib.util
import os

import pytest
import torch

import grouped_gemm_device_gb300 as g

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "moe_block_step", os.path.join(ROOT, "examples", "moe_block_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(block, x, dy, mask, coef):
    """The same block in fp64 with autograd; the experts are chosen by the block's own ids."""
    d = torch.float64
    leaf = {n: t.to(d).requires_grad_() for n, t in
            (("x", x), ("gamma", block.gamma), ("beta", block.beta), ("wr", block.wr),
             ("w1", block.w1), ("w2", block.w2), ("w_up", block.w_up), ("w_down", block.w_down))}
    h = torch.nn.functional.layer_norm(leaf["x"], (x.shape[1],), leaf["gamma"], leaf["beta"], 1e-5)
    logits = h @ leaf["wr"].t()
    ids = block.experts.topk_ids.long()
    E, k = logits.shape[1], ids.shape[1]
    w = torch.softmax(torch.gather(logits, 1, ids), dim=1)
    y = leaf["x"]
    F = leaf["w2"].shape[1]
    for e in range(E):
        z = h @ leaf["w1"][e]
        out = (torch.nn.functional.silu(z[:, :F]) * z[:, F:]) @ leaf["w2"][e]
        y = y + out * (w * (ids == e)).sum(dim=1, keepdim=True)
    z = h @ leaf["w_up"].t()
    y = y + (torch.nn.functional.silu(z[:, :block.S]) * z[:, block.S:]) @ leaf["w_down"].t()
    m = mask.to(d)
    n = m.sum()
    counts = torch.stack([((ids == e) & mask[:, None]).sum() for e in range(E)])
    p = (torch.softmax(logits, dim=1) * m[:, None]).sum(dim=0) / n
    aux = coef * (counts * E / (k * n) * p).sum()
    ((y * dy.to(d)).sum() + aux).backward()
    return y.detach(), aux.detach(), counts, {n: t.grad for n, t in leaf.items()}


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_step_matches_autograd(lib, example):
    torch.manual_seed(0)
    T, H, F, E, coef = 300, 128, 192, 4, 0.02
    block = example.MoEBlock(T, H, F, E, coef=coef, max_norm=1e9)
    x = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    dy = torch.randn(T, H, device="cuda").to(torch.bfloat16)
    mask = torch.rand(T, device="cuda") < 0.8
    y, aux, counts = block.forward(x, mask)
    y, aux, counts = y.clone(), aux.clone(), counts.clone()
    dx = block.backward(dy)
    ey, ea, ec, grad = reference(block, x, dy, mask, coef)
    assert counts.tolist() == ec.tolist()
    assert abs(float(aux) - float(ea)) <= 1e-2 * float(ea)       # logits from bf16 rows
    # bf16 rows (2^-8) throughout; the shared expert's products have two operands in E4M3, whose
    # rounding is 2.6% rms of a value: 3.7% of a product, 5% over two of them
    assert rel(y, ey) <= 0.06 and rel(dx, grad["x"]) <= 0.06
    got = {n: t.clone() for n, t in block.grads.items()}
    dw1 = torch.empty_like(block.w1)
    g.moe_pack_fc1_weight(got["w1p"], dw1, E, H, F, 1, 64, 1)
    got["w1"] = dw1
    for name in ("gamma", "beta", "wr", "w1", "w2", "w_up", "w_down"):
        assert rel(got[name], grad[name]) <= 0.08, name
    norm = sum(float(t.double().pow(2).sum()) for t in block.grads.values()) ** 0.5
    assert abs(float(block.grad_norm) - norm) <= 1e-5 * norm     # within the limit: not scaled


def test_clipped_gradients_have_the_limit_as_their_norm(lib, example):
    block = example.MoEBlock(64, 64, 64, 4, max_norm=0.5)
    x = torch.randn(64, 64, device="cuda").to(torch.bfloat16)
    for _ in range(2):  # the second step reuses the plan
        block.forward(x)
        block.backward(x)
        assert float(block.grad_norm) > 0.5
        norm = sum(float(t.double().pow(2).sum()) for t in block.grads.values()) ** 0.5
        assert abs(norm - 0.5) <= 0.5 * 2.0 ** -8


def test_example_runs(lib, example, capsys):
    example.main(["--tokens", "256", "--hidden", "128", "--ffn", "256", "--steps", "2"])
    out = capsys.readouterr().out
    assert out.count("step ") == 2 and "nan" not in out
