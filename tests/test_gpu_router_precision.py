"""The router loss's arithmetic beside its formula: exponentials of far logits, the reciprocal of a
row's sum, and the sums over blocks, each where fewer bits would show."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import block_ops as ob

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24        # half an ulp of fp32, relative
LEAST = 2.0 ** -149     # the smallest subnormal number


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def far_rows(T, E, lo, hi, seed=0):
    """Expert 0 at 0, the others at multiples of 1/8 in [lo, hi] below it, so that differences of
    logits are exact and, with hi <= -24, the other weights together are below half an ulp of 1."""
    r = np.random.default_rng([seed, T, E])
    x = r.integers(8 * lo, 8 * hi + 1, (T, E)).astype(np.float32) / np.float32(8)
    x[:, 0] = 0.0
    return x, np.zeros((T, 1), np.int32)


# exp: 2 ulp (4 units); the row's sum, its reciprocal and the product with it: one unit each; the
# mean over one token: one more
P_UNITS = 8


@pytest.mark.parametrize("E", [5, 64, 255, 256])
@pytest.mark.parametrize("lo,hi", [(-86, -24), (-103, -88)])
def test_probabilities_of_far_logits(lib, E, lo, hi):
    plan = g.RouterLoss(E, 1, 1)
    for seed in range(6):
        x, ids = far_rows(1, E, lo, hi, seed)
        p = plan.forward(dev(x), dev(ids))[2].double().cpu().numpy()
        want = ob.softmax(x.astype(np.float64))[0]
        assert (np.abs(p - want) <= P_UNITS * ULP * want + 2 * LEAST).all()


@pytest.mark.parametrize("E", [5, 64, 255, 256])
@pytest.mark.parametrize("lo,hi", [(-86, -24), (-103, -88)])
def test_gradient_of_far_logits(lib, E, lo, hi):
    """d = c p (f - s) with f = (E, 0, ..), s = E to half an ulp: beside p's units four roundings
    of the factors and of s."""
    T = 64
    x, ids = far_rows(T, E, lo, hi)
    plan = g.RouterLoss(E, 1, T, coef=float(T))
    plan.forward(dev(x), dev(ids))
    d = plan.backward(dev(x), dev(ids)).double().cpu().numpy()
    want, size = ob.router_grad(x.astype(np.float64), ids, float(T))
    assert (np.abs(d - want) <= (P_UNITS + 4) * ULP * size + 3 * E * LEAST).all()


def test_equal_logits_have_the_rounded_reciprocal(lib):
    """E equal weights of 1: a probability is fp32's 1 / E, every other step being exact."""
    for E in range(1, 257):
        plan = g.RouterLoss(E, 1, 1)
        x = torch.full((1, E), 0.75, device="cuda")
        p = plan.forward(x, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))[2]
        assert (p.cpu().numpy() == np.float32(1) / np.float32(E)).all(), E


def test_blocks_are_added_with_more_bits_than_a_block_has(lib):
    """One warp's worth of tokens an SM and warp. The first 32 put all weight on expert 0, the
    others 5.5e-8: 32 of those are less than half an ulp of 32, all of them together 35 ulp."""
    E, per = 256, 32
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = per * sms
    x = np.full((T, E), -40.0, np.float32)
    x[:per, 0] = 0.0
    x[per:, 1] = 0.0
    x[per:, 0] = np.log(5.5e-8)
    ids = np.zeros((T, 1), np.int32)
    plan = g.RouterLoss(E, 1, T, coef=1.0)
    loss, _, mean_prob = plan.forward(dev(x), dev(ids))
    want_loss, _, want, _, _ = ob.router_loss(x.astype(np.float64), ids, 1.0)
    # expert 0: exact ones, small terms to a few units of themselves, one sum rounded and divided
    assert abs(float(mean_prob[0].double()) - want[0]) <= 3 * ULP * want[0]
    assert abs(float(loss.double()) - want_loss) <= 4 * ULP * want_loss


@pytest.mark.parametrize("T", [25, 1000])
def test_loss_is_the_sum_of_its_terms(lib, T):
    """Against its own counts and mean probabilities in 64 bits. Seven experts, 32 apart, have terms
    just below half an ulp of expert 0's. mean_prob's rounding and the loss's own: 2 units."""
    E = 256
    x = np.full((T, E), -60.0, np.float32)
    x[:, 0] = 0.0
    x[:, 32::32] = -14.75
    ids = np.zeros((T, 1), np.int32)
    few = max(1, 68 * T // 1000)
    for i in range(1, 8):
        ids[(i - 1) * few:i * few] = 32 * i
    plan = g.RouterLoss(E, 1, T, coef=1.0)
    loss, counts, mean_prob = plan.forward(dev(x), dev(ids))
    f = counts.double() * E / T
    want = float((f * mean_prob.double()).sum())
    assert abs(float(loss.double()) - want) <= 2.5 * ULP * want
