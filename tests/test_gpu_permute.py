"""The layer under a given routing: the same as under its own, dropped slots, repeated experts."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
KINDS = [("bf16", 32), ("mxfp8", 128), ("nvfp4", 128)]


class Layer:
    def __init__(self, precision="bf16", align=32, T=300, E=6, k=3, H=256, F=256, seed=0, **kw):
        gen = torch.Generator().manual_seed(seed)

        def rand(*shape, scale=1.0):
            return (torch.randn(*shape, generator=gen) * scale).to(BF).cuda()

        self.T, self.E, self.k, self.H, self.F = T, E, k, H, F
        self.x, self.dy = rand(T, H), rand(T, H)
        self.w1 = rand(E, H, 2 * F, scale=0.05)
        self.w1p, self.w2 = g.pack_w1(self.w1), rand(E, F, H, scale=0.05)
        self.logits = torch.randn(T, E, generator=gen).cuda()
        self.layer = g.MoELayer(g.make_desc(E=E, k=k, H=H, F=F, T_max=T, precision=precision,
                                            align=align, rht_mask=0x1234, **kw))

    def results(self, T=None):
        T = self.T if T is None else T
        y = self.layer.forward(self.w1p, self.w2, T)
        outs = y, *self.layer.backward(self.dy[:T], self.w1p, self.w2, T)
        torch.cuda.synchronize()
        assert self.layer.device_error() == 0
        return [t.clone() for t in outs]


@pytest.mark.parametrize("precision,align", KINDS)
def test_same_as_the_layers_own_routing(lib, precision, align):
    a = Layer(precision, align)
    a.layer.route_permute(a.logits, a.x)
    ids, probs, counts = (t.clone() for t in (a.layer.topk_ids, a.layer.topk_probs, a.layer.counts))
    want = a.results()
    a.layer.counts.zero_()
    a.layer.ws.fill_(0)
    a.layer.permute(ids, probs, a.x)
    assert torch.equal(a.layer.counts, counts)
    assert all(torch.equal(p, q) for p, q in zip(want, a.results()))


@pytest.mark.parametrize("precision,align", KINDS)
def test_dropped_slots(lib, precision, align):
    """A token without slots gets y = dx = 0 and d_probs = 0; the others are as if it were not
    there."""
    a = Layer(precision, align)
    a.layer.route_permute(a.logits, a.x)
    ids, probs = a.layer.topk_ids.clone(), a.layer.topk_probs.clone()
    drop = torch.rand(a.T, generator=torch.Generator().manual_seed(1)).cuda() < 0.3
    ids[drop] = -1
    ids[5, 1], ids[6, 2] = a.E, -100
    a.layer.y.fill_(7.0)
    a.layer.permute(ids, probs, a.x)
    live = (ids >= 0) & (ids < a.E)
    assert torch.equal(a.layer.counts.cpu().long(),
                       torch.bincount(ids[live].cpu().long(), minlength=a.E))
    y, dx, dw1, dw2, dp = a.results()
    assert not y[drop].any() and not dx[drop].any() and not dp[~live].any()
    # the same tokens alone: token order and with it every row is the same
    keep = ~drop
    n = int(keep.sum())
    x, dy = a.x[keep].contiguous(), a.dy[keep].contiguous()
    a.layer.permute(ids[keep].contiguous(), probs[keep].contiguous(), x)
    a.dy = dy
    for p, q in zip((y[keep], dx[keep], dw1, dw2, dp[keep]), a.results(n)):
        assert torch.equal(p, q)
    row_of = torch.empty(n * a.k, dtype=torch.int32, device="cuda")
    g.moe_route_export(a.layer.desc, a.layer.ws, a.layer.ws_bytes, n, row_of=row_of)
    assert torch.equal(row_of.view(n, a.k) < 0, ~live[keep])


def test_against_fp64(lib):
    """Repeated experts (each slot its own row), dropped slots and weights of any sign, against the
    definition in 64 bits. Outputs are bf16 after bf16 stages (z, a): errors of about 2^-8 a stage,
    relative to the whole."""
    a = Layer(T=200, E=4, k=3, H=128, F=128)
    gen = torch.Generator().manual_seed(3)
    ids = torch.randint(-1, a.E + 1, (a.T, a.k), generator=gen, dtype=torch.int32).cuda()
    ids[:50] = 2
    probs = torch.randn(a.T, a.k, generator=gen).cuda()
    a.layer.permute(ids, probs, a.x)
    y, dx, _, dw2, dp = a.results()
    x, w1, w2 = (t.double().requires_grad_() for t in (a.x, a.w1, a.w2))
    p = probs.double().requires_grad_()
    out = torch.zeros(a.T, a.H, dtype=torch.float64, device="cuda")
    for j in range(a.k):
        for e in range(a.E):
            at = torch.nonzero(ids[:, j] == e)[:, 0]
            z = x[at] @ w1[e]
            act = torch.nn.functional.silu(z[:, :a.F]) * z[:, a.F:]
            out = out.index_add(0, at, p[at, j:j + 1] * (act @ w2[e]))
    want = torch.autograd.grad((out * a.dy.double()).sum(), (x, w2, p))
    for got, ref in ((y, out.detach()), (dx, want[0]), (dw2, want[1]), (dp, want[2])):
        assert float((got.double() - ref).norm() / ref.norm()) <= 4 * 2.0 ** -8


def test_every_slot_dropped_and_no_tokens(lib):
    a = Layer()
    none = torch.full((a.T, a.k), -1, dtype=torch.int32, device="cuda")
    probs = torch.ones(a.T, a.k, device="cuda")
    a.layer.permute(none, probs, a.x)
    assert not a.layer.counts.any()
    for t in a.results():
        assert not t.any()
    a.layer.permute(none[:0], probs[:0], a.x[:0])
    _, _, dw1, dw2, _ = a.results(0)
    assert not dw1.any() and not dw2.any()


def test_every_slot_on_one_expert(lib):
    a = Layer(T=257, k=3)
    ids = torch.full((a.T, a.k), a.E - 1, dtype=torch.int32, device="cuda")
    a.layer.permute(ids, torch.full((a.T, a.k), 0.5, device="cuda"), a.x)
    assert a.layer.counts.cpu().tolist() == [0] * (a.E - 1) + [a.T * a.k]
    three = a.results()[0]
    one = Layer(T=257, k=1)
    one.layer.permute(ids[:, :1].contiguous(), torch.full((a.T, 1), 1.5, device="cuda"), a.x)
    one.w1p, one.w2 = a.w1p, a.w2
    got = one.results()[0]
    # three rounded bf16 rows of half weight, added and rounded, against one of weight 1.5
    assert float((three.double() - got.double()).norm() / got.double().norm()) <= 3 * 2.0 ** -8


def test_in_a_graph(lib):
    a = Layer()
    plan = g.RouterTopK(a.E, a.k, a.T, score="sigmoid", scale=1.5)
    bias = torch.zeros(a.E, device="cuda")

    def step():
        ids, w, _ = plan.forward(a.logits, bias)
        a.layer.permute(ids, w, a.x)
        y = a.layer.forward(a.w1p, a.w2, a.T)
        return y, *a.layer.backward(a.dy, a.w1p, a.w2, a.T)

    step()
    bias[3] = 0.4
    want = [t.clone() for t in step()]
    bias.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    bias[3] = 0.4
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, outs))


def test_argument_checks(lib):
    a = Layer(T=16)
    ids = torch.zeros(16, 3, dtype=torch.int32, device="cuda")
    p = torch.zeros(16, 3, device="cuda")
    for args in ((ids.long(), p, a.x), (ids[:8], p, a.x), (ids, p.to(BF), a.x), (ids, p, a.x[:8]),
                 (ids, p, a.x.float()), (ids.cpu(), p, a.x), (ids, p, a.x, 17),
                 (ids, p, a.x[:, :128])):
        with pytest.raises(ValueError):
            a.layer.permute(*args)
    assert np.array_equal(ids.cpu().numpy(), np.zeros((16, 3), np.int32))


def test_first_weight_gradient_against_fp64(lib):
    """dW1 under repeated experts, dropped slots and weights of any sign, in its logical order: bf16 stages
    as in test_against_fp64."""
    a = Layer(T=200, E=4, k=3, H=128, F=128)
    gen = torch.Generator().manual_seed(3)
    ids = torch.randint(-1, a.E + 1, (a.T, a.k), generator=gen, dtype=torch.int32).cuda()
    ids[:50] = 2
    ids[ids == 3] = -1                              # an expert without rows
    probs = torch.randn(a.T, a.k, generator=gen).cuda()
    a.layer.permute(ids, probs, a.x)
    dw1 = a.results()[2]
    got = torch.empty_like(a.w1)
    g.moe_pack_fc1_weight(dw1, got, a.E, a.H, a.F, 1, 64, 1)
    x, w1, w2, p = a.x.double(), a.w1.double().requires_grad_(), a.w2.double(), probs.double()
    out = torch.zeros(a.T, a.H, dtype=torch.float64, device="cuda")
    for j in range(a.k):
        for e in range(a.E):
            at = torch.nonzero(ids[:, j] == e)[:, 0]
            z = x[at] @ w1[e]
            act = torch.nn.functional.silu(z[:, :a.F]) * z[:, a.F:]
            out = out.index_add(0, at, p[at, j:j + 1] * (act @ w2[e]))
    (want,) = torch.autograd.grad((out * a.dy.double()).sum(), w1)
    assert float((got.double() - want).norm() / want.norm()) <= 4 * 2.0 ** -8
    assert not got[3].any()
