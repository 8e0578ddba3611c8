"""The choice of experts and the gradient of its weights against the fp64 oracle."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import step_ops as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24   # half a step of fp32


def f64(t):
    return t.detach().double().cpu().numpy()


def make(T, E, dtype=F32, seed=0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=gen) * spread).to(dtype).cuda()


def check_forward(x, bias, mask, k, score, groups, of, top, renorm, scale=2.5):
    T, E = x.shape
    plan = g.RouterTopK(E, k, T + 3, score=score, n_group=groups, topk_group=of, group_top=top,
                        renorm=renorm, scale=scale, dtype=x.dtype)
    ids, w, counts = (t.cpu().numpy() for t in plan.forward(x, bias, mask))
    b = None if bias is None else f64(bias)
    m = None if mask is None else mask.cpu().numpy().astype(bool)
    want, ww, margin = so.route(f64(x), k, score, b, m, groups, of, top, renorm, scale)
    # fp32 values up to 2 (scores up to 1 and biases of order 1, and sums of two) are off by a few
    # half steps of 2: tokens with two deciding values nearer than that may choose otherwise; they are
    # few (32 U times the values' density, which is at most some thousands)
    clear = margin > 32 * U
    assert (~clear).sum() <= max(1, 0.03 * T) and (ids[clear] == want[clear]).all()
    # the others choose different experts of the same number
    for t in np.flatnonzero(~clear):
        assert len(set(ids[t])) == k and (ids[t] >= 0).all() and (ids[t] < E).all()
    # exp off by two steps (4 U) at most and by U of its argument's magnitude; 1 + e, its reciprocal,
    # the sum of eight and its epsilon (4 additions deep), the quotient and the scale: 1 each. In
    # subnormal scores a step is absolute
    reach = np.abs(f64(x)[np.isfinite(f64(x))]).max(initial=0) * 2
    tol = (24 + reach) * U
    assert (np.abs(w - ww)[clear] <= tol * np.abs(ww)[clear] + 1e-37 * scale).all()
    live = np.ones(T, bool) if m is None else m
    assert (ids[~live] == -1).all() and not w[~live].any()
    assert (counts == np.bincount(ids[live].reshape(-1), minlength=E)).all()
    return plan


SHAPES = [(1, 1, 1, 1, 1), (5, 2, 1, 1, 1), (64, 8, 2, 1, 1), (33, 7, 7, 1, 1), (100, 256, 8, 8, 4),
          (77, 60, 4, 1, 1), (50, 33, 3, 11, 5), (40, 160, 6, 8, 3), (300, 128, 4, 1, 1),
          (9, 255, 8, 5, 2), (21, 6, 2, 3, 1), (17, 240, 8, 240, 8), (65, 64, 8, 4, 2),
          (31, 16, 8, 8, 4), (1000, 256, 1, 1, 1)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_forward(lib, shape, score, renorm):
    T, E, k, groups, of = shape
    for dtype in (F32, BF):
        x = make(T, E, dtype, seed=T, spread=2.0)
        bias = make(1, E, seed=1, spread=0.3)[0]
        mask = torch.rand(T, generator=torch.Generator().manual_seed(2)).cuda() < 0.8
        tops = (1, 2) if E // groups > 1 else (1,)
        for top in tops:
            check_forward(x, None, None, k, score, groups, of, top, renorm)
            check_forward(x, bias, mask, k, score, groups, of, top, renorm)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_ties_go_to_the_lower_index(lib, score):
    x = torch.zeros(4, 256, device="cuda")
    x[1, 200:] = 1.0
    x[2] = (torch.arange(256) % 2).float()
    x[3, 5] = -0.0
    plan = g.RouterTopK(256, 8, 4, score=score)
    ids = plan.forward(x)[0].cpu().tolist()
    assert ids[0] == list(range(8)) and ids[1] == list(range(200, 208))
    assert ids[2] == list(range(1, 16, 2)) and ids[3] == list(range(8))
    plan = g.RouterTopK(256, 8, 4, score=score, n_group=8, topk_group=2, group_top=2)
    ids = plan.forward(x, torch.zeros(256, device="cuda"))[0].cpu().tolist()
    assert ids[0] == list(range(8)) and ids[1] == list(range(200, 208))
    assert ids[2] == list(range(1, 16, 2))
    # quantised logits: every row has ties, the oracle breaks them the same way
    gen = torch.Generator().manual_seed(3)
    q = (torch.randint(-3, 4, (200, 64), generator=gen).float() / 2).cuda()
    for bias in (None, torch.zeros(64, device="cuda")):
        check_forward(q, bias, None, 8, score, 8, 4, 2, True)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_logits_that_are_not_finite(lib, score, renorm):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[0.5, -inf, 1.0, nan], [-inf] * 4, [nan] * 4, [inf, 1.0, inf, -inf],
                      [3e38, -3e38, 0.0, 1.0], [-200.0, -100.0, -300.0, -400.0]], device="cuda")
    plan = g.RouterTopK(4, 2, 6, score=score, renorm=renorm)
    ids, w, counts = plan.forward(x)
    want, ww, _ = so.route(f64(x), 2, score, renorm=renorm)
    assert (ids.cpu().numpy() == want).all() and int(counts.sum()) == 12
    # exp(200) and exp(100) are beyond fp32's range: a score below 2^-128 is 0, which a sum of 1e-20
    # divides by (and 1 without renorm). A softmax's exp has absolute steps of 2^-149 there
    low = 2.0 ** -128 / 1e-20 if score == "sigmoid" else 2.0 ** -148
    assert (np.abs(f64(w) - ww) <= 30 * U * np.abs(ww) + low).all()
    # a bias of -inf shuts an expert out, one of +inf lets it in, NaN reads as -inf
    bias = torch.tensor([-inf, 0.0, inf, nan], device="cuda")
    ids = g.RouterTopK(4, 2, 6, score=score).forward(torch.zeros(6, 4, device="cuda"), bias)[0]
    assert ids.cpu().tolist() == [[2, 1]] * 6
    ids = g.RouterTopK(4, 4, 6, score=score).forward(torch.zeros(6, 4, device="cuda"), bias)[0]
    assert ids.cpu().tolist() == [[2, 1, 0, 3]] * 6


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,of", [(256, 8, 4), (256, 1, 1), (64, 4, 2), (40, 1, 1)])
def test_biases_of_any_size(lib, score, E, groups, of):
    """Biases far beyond the scores, infinite ones among them, and logits so near to one another that
    most choices are close: fp32 sums, of which many are equal, and the lower index then."""
    gen = torch.Generator().manual_seed(E)
    x = torch.randn(200, E, generator=gen).cuda()
    x[50:100] *= 1e-6
    x[100:150] *= 30
    x[150:] = x[150:].round()
    inf = float("inf")
    for scale in (1e-7, 1.0, 100.0, 1e6):
        bias = (torch.randn(E, generator=gen) * scale).cuda()
        for special in (False, True):
            if special:
                bias[3], bias[7], bias[8], bias[20] = inf, -inf, inf, float("nan")
            for top in ((1, 2) if groups > 1 else (1,)):
                plan = g.RouterTopK(E, 8, 200, score=score, n_group=groups, topk_group=of,
                                    group_top=top)
                ids = plan.forward(x, bias)[0]
                assert torch.equal(ids.long(), by_steps(x, bias, score, 8, groups, of, top))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
def test_groups_that_nearly_tie(lib, score, top):
    """Two groups of the same values but for a few steps of fp32, elsewhere nothing near: as many groups
    stay as should, and the right one of the two."""
    gen = torch.Generator().manual_seed(top)
    T, E, groups = 3000, 64, 4
    x = torch.randn(T, E, generator=gen)
    x[:, 48:] = x[:, 16:32] * (1 + torch.randint(-3, 4, (T, 16), generator=gen) * 2.0 ** -23)
    bias = torch.randn(E, generator=gen) * 0.1
    bias[48:] = bias[16:32]
    x, bias = x.cuda(), bias.cuda()
    for of in (1, 2, 3):
        plan = g.RouterTopK(E, 8, T, score=score, n_group=groups, topk_group=of, group_top=top)
        ids = plan.forward(x, bias)[0].long()
        assert torch.equal(ids, by_steps(x, bias, score, 8, groups, of, top))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("top", [1, 2])
def test_groups_with_infinite_biases(lib, score, top):
    """Experts shut out or forced in: groups of one open expert, of none, of several forced ones."""
    gen = torch.Generator().manual_seed(top)
    T, E, groups, inf = 64, 64, 8, float("inf")
    x = torch.randn(T, E, generator=gen).cuda()
    biases = []
    for fill in (-inf, 0.0):
        for n in (3, 20):
            b = torch.full((E,), fill)
            b[torch.randperm(E, generator=gen)[:n]] = torch.randn(n, generator=gen)
            b[torch.randperm(E, generator=gen)[:n]] = -inf if fill == 0.0 else 0.5
            biases += [b, torch.where(torch.rand(E, generator=gen) < 0.1, inf, b)]
    for b in biases:
        b = b.cuda()
        for of in (1, 3, 7):
            plan = g.RouterTopK(E, 8, T, score=score, n_group=groups, topk_group=of, group_top=top)
            ids = plan.forward(x, b)[0].long()
            assert torch.equal(ids, by_steps(x, b, score, 8, groups, of, top))


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_many_tokens(lib, score):
    """Many tokens a warp, every choice as the definition's single steps."""
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(40_000, 256, generator=gen).cuda()
    bias = (0.1 * torch.randn(256, generator=gen)).cuda()
    plan = g.RouterTopK(256, 8, 40_000, score=score, n_group=8, topk_group=4, group_top=2)
    assert torch.equal(plan.forward(x, bias)[0].long(), by_steps(x, bias, score, 8, 8, 4, 2))


def by_steps(x, bias, score, k, groups, of, top):
    """The definition in single fp32 operations of torch, on the GPU."""
    T, E = x.shape
    if score == "sigmoid":
        s = torch.reciprocal(1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        total = torch.nn.functional.pad(e, (0, (1 << (E - 1).bit_length()) - E))
        while total.shape[1] > 1:
            total = total[:, 0::2] + total[:, 1::2]
        s = e * torch.reciprocal(total)
    v = s + torch.where(bias.isnan(), -torch.inf, bias)
    if groups > 1:
        best = v.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :top].sum(2)
        best = torch.where(best.isnan(), -torch.inf, best)
        kept = best.sort(dim=1, descending=True, stable=True).indices[:, :of]
        keep = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        keep = keep.repeat_interleave(E // groups, 1)
        # an expert of a kept group at -inf comes before those of other groups
        order = torch.where(keep, v, -torch.inf).sort(dim=1, descending=True, stable=True).indices
        inside = keep.gather(1, order)
        order = order.gather(1, (~inside).int().sort(dim=1, stable=True).indices)
        return order[:, :k]
    return v.sort(dim=1, descending=True, stable=True).indices[:, :k]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_backward(lib, shape, score, renorm):
    T, E, k = shape[:3]
    gen = torch.Generator().manual_seed(T + 1)
    for dtype in (F32, BF):
        x = make(T, E, dtype, seed=T, spread=2.0)
        dw = torch.randn(T, k, generator=gen).cuda()
        ids = torch.topk(torch.rand(T, E, generator=gen), k, dim=1).indices.int()
        ids[::4] = -1
        if T > 8:
            ids[5] = E                      # out of range: dropped
            ids[6, 0] = -7
            ids[7] = ids[7, 0].item()       # one expert in every slot
        add = torch.randn(T, E + 5, generator=gen).cuda()[:, :E]
        plan = g.RouterTopK(E, k, T + 2, score=score, renorm=renorm, scale=1.5, dtype=dtype)
        d, mag = so.route_grad(f64(x), ids.numpy(), f64(dw), score, renorm, 1.5)
        # as the weights', the products, a sum of 256 products in a tree of 8 + 8 additions
        reach = np.abs(f64(x)).max() * 2
        tol = (50 + reach) * U * mag + 2.0 ** -140
        got = f64(plan.backward(x, dw, ids.cuda()))
        assert (np.abs(got - d) <= tol).all()
        keep = add.clone()
        got = f64(plan.backward(x, dw, ids.cuda(), add_to=add))
        assert (np.abs(got - d - f64(add)) <= tol + U * np.abs(f64(add) + d) * 1.01).all()
        assert torch.equal(add, keep)


@pytest.mark.parametrize("E", [3, 16, 40, 256])
@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
def test_a_single_slot_renormalised(lib, E, score):
    """Its weight is 1 whatever the logit: what is left of the gradient is u less its rounded self, times
    the slope over the score, for a sigmoid; 0 for a softmax."""
    x, dw = make(300, E, spread=2.0), make(300, 1, seed=1)
    ids = torch.randint(0, E, (300, 1), generator=torch.Generator().manual_seed(2)).int().cuda()
    plan = g.RouterTopK(E, 1, 300, score=score, scale=2.5)
    d = f64(plan.backward(x, dw, ids))
    # u s / S and u are a rounding of each apart at most, divided by s; the slope over s is at most 1
    most = 2 * U * 2.5 * np.abs(f64(dw)) if score == "sigmoid" else 0.0
    assert (np.abs(d) <= most * 1.01).all()


def test_backward_in_place_and_strides(lib):
    x = make(50, 40)
    wide = torch.full((50, 64), 7.0, device="cuda")
    wide[:, 3:43] = x
    plan = g.RouterTopK(40, 4, 50)
    ids, w, _ = (t.clone() for t in plan.forward(x))
    assert all(torch.equal(a, b) for a, b in zip((ids, w), plan.forward(wide[:, 3:43])))
    dw = make(50, 4, seed=5)
    d = plan.backward(x, dw).clone()
    assert torch.equal(plan.backward(wide[:, 3:43], dw, ids), d)
    base = make(50, 40, seed=6)
    want = base + d
    g.moe_router_topk_bwd(x, 40, 1, ids, dw, 50, 40, 4, 1, 1, 1.0, base, 40, base, 40)
    assert torch.equal(base, want)


def test_empty_and_masked_batches(lib):
    plan = g.RouterTopK(8, 2, 16)
    plan.counts.fill_(5)
    ids, w, counts = plan.forward(torch.empty(0, 8, device="cuda"))
    assert ids.shape == (0, 2) and not counts.any()
    mask = torch.zeros(16, dtype=torch.bool, device="cuda")
    ids, w, counts = plan.forward(make(16, 8), token_mask=mask)
    assert (ids == -1).all() and not w.any() and not counts.any()
    assert not plan.backward(make(16, 8), make(16, 2)).any()


def test_rows_behind_the_last_token_stay(lib):
    plan = g.RouterTopK(8, 2, 16)
    plan.topk_ids.fill_(77)
    plan.topk_weights.fill_(7.0)
    plan.forward(make(5, 8))
    assert (plan.topk_ids[5:] == 77).all() and (plan.topk_weights[5:] == 7).all()


def test_same_results_again_in_a_graph_and_on_another_stream(lib):
    x, bias, dw = make(3000, 256), make(1, 256, seed=1)[0], make(3000, 8, seed=2)
    plan = g.RouterTopK(256, 8, 3000, n_group=8, topk_group=4, group_top=2, scale=2.5)

    def call():
        return (*plan.forward(x, bias), plan.backward(x, dw))

    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = call()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    for stream in (s, s.cuda_stream):
        plan.forward(x, bias, stream=stream)
        s.synchronize()
        assert torch.equal(plan.topk_ids, want[0])


def test_argument_checks(lib):
    plan = g.RouterTopK(8, 2, 16)
    x, dw = torch.zeros(16, 8, device="cuda"), torch.zeros(16, 2, device="cuda")
    bad = [lambda: plan.backward(x, dw)]        # no forward yet
    for f in bad:
        with pytest.raises(ValueError):
            f()
    plan.forward(x[:4])
    ids = torch.zeros(16, 2, dtype=torch.int32, device="cuda")
    for f in (lambda: plan.backward(x, dw), lambda: plan.forward(x.to(BF)),
              lambda: plan.forward(x.cpu()), lambda: plan.forward(x[:, :4]),
              lambda: plan.forward(torch.zeros(17, 8, device="cuda")),
              lambda: plan.forward(x, torch.zeros(8, device="cuda", dtype=BF)),
              lambda: plan.forward(x, torch.zeros(7, device="cuda")),
              lambda: plan.forward(x, None, torch.ones(16, device="cuda")),
              lambda: plan.forward(x, None, torch.ones(15, device="cuda").bool()),
              lambda: plan.backward(x, dw[:8], ids), lambda: plan.backward(x, dw.to(BF), ids),
              lambda: plan.backward(x, dw, ids.long()), lambda: plan.backward(x, dw, ids[:8]),
              lambda: plan.backward(x, dw, ids, add_to=x[:8]),
              lambda: plan.backward(x, dw, ids, add_to=x.to(BF)),
              lambda: g.RouterTopK(8, 2, 16, score="tanh"),
              lambda: g.RouterTopK(8, 2, 16, dtype=torch.float16)):
        with pytest.raises(ValueError):
            f()
    for kw in (dict(n_group=3), dict(n_group=4, topk_group=5), dict(n_group=8, group_top=2)):
        with pytest.raises(g.MoeError):
            g.RouterTopK(8, 2, 16, **kw).forward(x)
