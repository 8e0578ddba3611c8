"""The classes around the operators: their checks of arguments, and buffers larger than a call."""
import pytest
import torch

import grouped_gemm_device_gb300 as g

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def raises(fn, *args, **kw):
    with pytest.raises(ValueError):
        fn(*args, **kw)


def test_router_loss_checks(lib):
    plan = g.RouterLoss(8, 2, 16)
    lg, ids = torch.zeros(16, 8, device="cuda"), torch.zeros(16, 2, dtype=torch.int32).cuda()
    plan.forward(lg, ids)
    raises(plan.forward, lg.cpu(), ids)
    raises(plan.forward, lg.to(BF), ids)
    raises(plan.forward, lg, ids.long())
    raises(plan.forward, lg, ids[:8])
    raises(plan.forward, lg[:, :4], ids)
    raises(plan.forward, lg.t().contiguous().t(), ids)
    raises(plan.forward, lg, ids, torch.ones(16, device="cuda"))
    raises(plan.forward, torch.zeros(17, 8, device="cuda"), torch.zeros(17, 2).int().cuda())
    raises(plan.backward, lg, ids, torch.zeros(16, 3, device="cuda"))
    raises(plan.backward, lg, ids, d_loss=torch.zeros(2, device="cuda"))
    with pytest.raises(g.MoeError):  # one of the pair is missing
        plan.backward(lg, ids, torch.zeros(16, 2, device="cuda"))


def test_layernorm_checks(lib):
    ln = g.LayerNorm(64, 8)
    x, w = torch.zeros(8, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")
    ln.forward(x, w, w)
    raises(ln.forward, x.float())
    raises(ln.forward, x.cpu())
    raises(ln.forward, x[0])
    raises(ln.forward, x, w.float())
    raises(ln.forward, x, w[:32])
    raises(ln.forward, torch.zeros(9, 64, dtype=BF, device="cuda"))
    raises(ln.backward, x[:4], x)
    raises(ln.backward, x, x, mean=torch.zeros(4, device="cuda"))
    raises(g.LayerNorm, 64, 8, dtype=torch.float16)


def test_grad_clip_checks(lib):
    t = torch.zeros(8, 4, device="cuda")
    raises(g.GradClip, [t.t()])
    raises(g.GradClip, [t.cpu()])
    raises(g.GradClip, [t], [t, t])
    raises(g.GradClip, [t], [t.to(BF)])
    raises(g.GradClip, [t.half()])
    with pytest.raises(g.MoeError):
        g.GradClip([t]).clip(0.0)


def test_fp8_linear_checks(lib):
    lin = g.Fp8Linear(32, 64, 8)
    x, w = torch.zeros(8, 64, dtype=BF, device="cuda"), torch.zeros(32, 64, dtype=BF, device="cuda")
    raises(lin.forward, x)          # no weight yet
    raises(lin.set_weight, w.t())
    raises(lin.set_weight, w.float())
    lin.set_weight(w)
    raises(lin.backward, torch.zeros(8, 32, dtype=BF, device="cuda"))  # no forward yet
    raises(lin.forward, x.cpu())
    raises(lin.forward, x[:, :32])
    raises(lin.forward, torch.zeros(9, 64, dtype=BF, device="cuda"))
    lin.forward(x[:4])
    raises(lin.backward, torch.zeros(8, 32, dtype=BF, device="cuda"))  # other rows
    infer = g.Fp8Linear(32, 64, 8, train=False)
    infer.set_weight(w)
    infer.forward(x)
    raises(infer.backward, torch.zeros(8, 32, dtype=BF, device="cuda"))


def test_calls_smaller_than_the_buffers(lib):
    """Results of a part of the rows equal those of a class made for that part."""
    gen = torch.Generator().manual_seed(0)
    x = torch.randn(50, 96, generator=gen).to(BF).cuda()
    w = (0.02 * torch.randn(40, 96, generator=gen)).to(BF).cuda()
    dy = torch.randn(50, 40, generator=gen).to(BF).cuda()
    big, small = g.Fp8Linear(40, 96, 300), g.Fp8Linear(40, 96, 50)
    outs = []
    for lin in (big, small):
        lin.set_weight(w)
        outs.append([t.clone() for t in (lin.forward(x), *lin.backward(dy))])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    lg = torch.randn(50, 8, generator=gen).cuda()
    ids = torch.topk(lg, 2).indices.int()
    outs = []
    for plan in (g.RouterLoss(8, 2, 300), g.RouterLoss(8, 2, 50)):
        outs.append([t.clone() for t in (*plan.forward(lg, ids), plan.backward(lg, ids))])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    outs = []
    for ln in (g.LayerNorm(96, 300), g.LayerNorm(96, 50)):
        outs.append([t.clone() for t in (*ln.forward(x), *ln.backward(x, x))])
    assert all(torch.equal(a, b) for a, b in zip(*outs))
