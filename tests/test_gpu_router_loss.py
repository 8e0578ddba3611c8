"""Router balance loss and logit gradient against the fp64 oracle and against differences."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import block_ops as ob

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24


def make(T, E, k, seed=0, mask=False, bias=1.1):
    r = np.random.default_rng([seed, T, E, k])
    lg = r.standard_normal((T, E)).astype(np.float32)
    lg -= (bias * np.log(r.permutation(E) + 1.0)).astype(np.float32)
    ids = np.argsort(-lg, axis=1, kind="stable")[:, :k].astype(np.int32)
    w = np.exp(np.take_along_axis(lg, ids.astype(np.int64), axis=1))
    w = (w / w.sum(axis=1, keepdims=True)).astype(np.float32)
    dw = (1e-3 * r.standard_normal((T, k))).astype(np.float32)
    m = r.random(T) < 0.7 if mask else None
    return lg, ids, w, dw, m


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(lg, ids, w, dw, m, coef=0.02, d_loss=1.5, logits_dev=None):
    T, E = lg.shape
    plan = g.RouterLoss(E, ids.shape[1], T, coef=coef)
    x = dev(lg) if logits_dev is None else logits_dev
    loss, counts, mean_prob = plan.forward(x, dev(ids), dev(m))
    dl = plan.backward(x, dev(ids), dev(w), dev(dw), dev(m), torch.tensor([d_loss]).cuda())
    torch.cuda.synchronize()
    el, ec, em, _, n = ob.router_loss(lg, ids, coef, m)
    assert counts.cpu().numpy().tolist() == ec.tolist()
    assert int(plan.n_valid) == n
    # p: exp within 2 ulp of an argument within 1/2 ulp of |x - max| <= 32, sums of <= 256 terms
    # in trees, one product: 64 ulp covers them; the means add at most T/32 terms in a row
    np.testing.assert_allclose(mean_prob.cpu().numpy(), em, rtol=(64 + T / 32) * ULP, atol=0)
    assert abs(float(loss) - el) <= (64 + T / 32) * ULP * abs(el)
    ed, size = ob.router_grad(lg, ids, coef, m, d_loss, w, dw)
    err = np.abs(dl.cpu().numpy() - ed)
    assert (err <= 80 * ULP * size + 1e-42).all(), float((err - 80 * ULP * size).max())
    return dl


@pytest.mark.parametrize("E,k", [(1, 1), (2, 1), (3, 2), (4, 2), (7, 3), (8, 2), (16, 4), (31, 8),
                                 (64, 6), (100, 8), (130, 5), (254, 8), (255, 8), (256, 8)])
@pytest.mark.parametrize("T,mask", [(1, False), (33, True), (1000, True)])
def test_matches_oracle(lib, T, E, k, mask):
    check(*make(T, E, k, mask=mask))


def test_many_tokens(lib):
    check(*make(20000, 32, 4, mask=True))


def test_row_stride_and_unaligned_rows(lib):
    lg, ids, w, dw, m = make(257, 12, 3, mask=True)
    for pad, shift in ((4, 0), (5, 0), (4, 1)):
        buf = torch.full((257 * (12 + pad) + 4,), float("nan"), device="cuda")
        x = buf[shift:shift + 257 * (12 + pad)].view(257, 12 + pad)[:, :12]
        x.copy_(dev(lg))
        check(lg, ids, w, dw, m, logits_dev=x)


def test_no_valid_token(lib):
    lg, ids, w, dw, _ = make(40, 8, 2)
    m = np.zeros(40, bool)
    plan = g.RouterLoss(8, 2, 40)
    plan.loss.fill_(7), plan.counts.fill_(7), plan.mean_prob.fill_(7)
    loss, counts, mean_prob = plan.forward(dev(lg), dev(ids), dev(m))
    assert float(loss) == 0 and not counts.any() and not mean_prob.any()
    d = plan.backward(dev(lg), dev(ids), token_mask=dev(m))
    assert not d.any()
    # the routing probabilities' part does not depend on the mask
    check(lg, ids, w, dw, m)


def test_no_token(lib):
    plan = g.RouterLoss(8, 2, 4)
    loss, counts, _ = plan.forward(torch.empty(0, 8).cuda(), torch.empty(0, 2).int().cuda())
    assert float(loss) == 0 and not counts.any()
    assert plan.backward(torch.empty(0, 8).cuda(), torch.empty(0, 2).int().cuda()).shape == (0, 8)


def test_infinite_and_nan_logits(lib):
    lg, ids, w, dw, m = make(64, 24, 4, mask=True)
    lg[3] = -np.inf                    # a row whose experts are all masked: uniform
    lg[4, 5:] = -np.inf
    lg[5, 2] = np.inf                  # takes all the weight
    lg[6, 1] = lg[6, 9] = np.inf       # share it
    lg[7, 0] = np.nan                  # reads as -inf
    lg[8] = -3.4028235e38              # a mask of the type's lowest value
    lg[9, 1:] = -3.4028235e38
    check(lg, ids, w, dw, m)


def test_dropped_slots_count_nowhere(lib):
    lg, ids, w, dw, m = make(200, 16, 4, mask=True)
    r = np.random.default_rng(5)
    ids[r.random(ids.shape) < 0.3] = -1
    ids[0] = 16
    check(lg, ids, w, dw, m)


def test_loss_alone_and_default_upstream(lib):
    lg, ids, w, dw, m = make(100, 10, 2, mask=True)
    plan = g.RouterLoss(10, 2, 100, coef=0.5)
    plan.forward(dev(lg), dev(ids), dev(m))
    d = plan.backward(dev(lg), dev(ids), token_mask=dev(m)).cpu().numpy()
    ed, size = ob.router_grad(lg, ids, 0.5, m)
    assert (np.abs(d - ed) <= 80 * ULP * size).all()


def test_gradient_against_differences(lib):
    """The loss has fp32 results; central differences of step 2^-6 in the logits, where the
    truncation error (third derivatives of a softmax are below 1) is step^2 / 6 and the rounding
    error 2 ulp of the loss over the step."""
    T, E, k, coef = 6, 5, 2, 1.0
    lg, ids, *_ = make(T, E, k, bias=0.3)
    plan = g.RouterLoss(E, k, T, coef=coef)
    h = 2.0 ** -6
    plan.forward(dev(lg), dev(ids))
    d = plan.backward(dev(lg), dev(ids)).cpu().numpy().copy()
    fmax = E / 1.0
    for t in range(T):
        for e in range(E):
            vals = []
            for s in (h, -h):
                z = lg.copy()
                z[t, e] += np.float32(s)
                vals.append(float(plan.forward(dev(z), dev(ids))[0].double()))
            num = (vals[0] - vals[1]) / (2 * h)
            assert abs(num - d[t, e]) <= fmax / T * h * h / 6 + 4 * ULP * 2.0 / h


def test_same_bits_again_and_on_another_stream(lib):
    lg, ids, w, dw, m = make(5000, 64, 6, mask=True)
    x, i, mm, ww, dd = dev(lg), dev(ids), dev(m), dev(w), dev(dw)
    plan = g.RouterLoss(64, 6, 5000)

    def once(stream=None):
        loss, c, p = plan.forward(x, i, mm, stream=stream)
        d = plan.backward(x, i, ww, dd, mm, stream=stream)
        return loss.clone(), c.clone(), p.clone(), d.clone()

    first = once()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = once()
    s.synchronize()
    for a, b, c in zip(first, other, once()):
        assert torch.equal(a, b) and torch.equal(a, c)


def test_graph_capture(lib):
    lg, ids, w, dw, m = make(3000, 8, 2, mask=True)
    x, i, mm, ww, dd = dev(lg), dev(ids), dev(m), dev(w), dev(dw)
    plan = g.RouterLoss(8, 2, 3000, coef=0.02)
    plan.forward(x, i, mm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.forward(x, i, mm)
        d = plan.backward(x, i, ww, dd, mm)
    lg2 = lg[::-1].copy()
    x.copy_(dev(lg2))
    graph.replay()
    torch.cuda.synchronize()
    ed, size = ob.router_grad(lg2, ids, 0.02, m, 1.0, w, dw)
    assert (np.abs(d.cpu().numpy() - ed) <= 80 * ULP * size + 1e-42).all()


@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (3, 3), (6, 5), (8, 8), (64, 8), (256, 8)])
def test_slots_that_share_an_expert(lib, E, k):
    """Ids that repeat, all of them or some, invalid ones among them: summed in their order."""
    lg, ids, w, dw, m = make(777, E, k, mask=True)
    r = np.random.default_rng(E)
    ids[::3] = r.integers(0, E, (len(ids[::3]), 1))           # one expert for every slot
    ids[1::3] = r.integers(-1, E, (len(ids[1::3]), k))
    first = check(lg, ids, w, dw, m)
    again = check(lg, ids, w, dw, m)
    assert torch.equal(first, again)
