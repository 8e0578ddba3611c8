"""Global gradient norm and clipping against the fp64 oracle."""
import math

import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import block_ops as ob

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


def f64(t):
    return t.detach().double().cpu().numpy()


def make(sizes, types, seed=0, scale=1e-2):
    gen = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=gen) * scale).to(t).cuda() for n, t in zip(sizes, types)]


def check(grads, max_norm, in_place):
    want = [f64(t) for t in grads]
    norm, c = ob.clip(want, max_norm)
    outs = None if in_place else [torch.full_like(t, 7.0) for t in grads]
    plan = g.GradClip(grads, outs)
    got = plan.clip(max_norm)
    torch.cuda.synchronize()
    # fp32 runs of 32 squares (at most 36 roundings of partial sums), fp64 beyond, one rounding
    # of the root; the factor's two operations and its product with an element
    assert abs(float(got.double()) - norm) <= norm * 20 * 2.0 ** -24
    for w, o in zip(want, plan.outs):
        err = np.abs(f64(o) - w * c)
        assert (err <= np.abs(w * c) * (HALF[o.dtype] * 1.01 + 24 * 2.0 ** -24) + 2.0 ** -134).all()
    if not in_place:
        for w, t in zip(want, grads):
            assert (f64(t) == w).all()
    return plan


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("frac", [0.25, 3.0])
@pytest.mark.parametrize("sizes", [[1], [5], [4096], [4097, 1, 0, 33], [100003, 7, 65536, 129],
                                   [3_000_001, 12]])
def test_matches_oracle(lib, sizes, frac, in_place):
    for types in ([BF] * len(sizes), [F32] * len(sizes), [BF, F32] * len(sizes)):
        grads = make(sizes, types)
        norm, _ = ob.clip([f64(t) for t in grads], 1.0)
        check(grads, frac * norm, in_place)


@pytest.mark.parametrize("dt,step", [(BF, 2), (F32, 4)])
def test_views_off_16_byte_boundaries(lib, dt, step):
    """Parameters packed into one flat buffer: each starts wherever the last one ended; outs
    with another offset than their gradients."""
    sizes = [3, 17, 1000, 8191, 1, 2, 300_007]
    flat = make([sum(sizes)], [dt])[0]
    keep = flat.clone()
    grads, at = [], 0
    for n in sizes:
        grads.append(flat[at:at + n])
        at += n
    assert any(t.data_ptr() % 16 for t in grads)
    norm, c = ob.clip([f64(keep)], 0.1)
    check([t.clone() for t in grads], 0.1, False)
    obuf = torch.full((at + 16,), 5.0, dtype=dt, device="cuda")
    outs, at = [], 1
    for n in sizes:
        outs.append(obuf[at:at + n])
        at += n
    g.GradClip(grads, outs).clip(0.1)
    err = np.abs(f64(obuf[1:at]) - f64(keep) * c)
    assert (err <= np.abs(f64(keep) * c) * (HALF[dt] * 1.01 + 24 * 2.0 ** -24) + 2.0 ** -134).all()
    assert (obuf[0] == 5).all() and (obuf[at:] == 5).all()
    g.GradClip(grads).clip(0.1)                      # in place in the flat buffer
    assert torch.equal(flat, obuf[1:at])


def test_many_tensors(lib):
    sizes = [(i * 37) % 501 for i in range(700)]
    check(make(sizes, [BF, F32] * 350), 0.05, True)
    check(make(sizes, [BF, F32] * 350), 0.05, False)


def test_within_the_limit_nothing_changes(lib):
    grads = make([1000, 3001], [BF, F32])
    keep = [t.clone() for t in grads]
    plan = g.GradClip(grads)
    norm = float(plan.clip(1e3))
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))
    assert norm == float(plan.clip(math.inf))
    assert all(torch.equal(a, b) for a, b in zip(keep, grads))


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e15, 1e25])
def test_magnitudes_whose_squares_leave_fp32(lib, scale):
    grads = make([5000, 77], [F32, BF], scale=scale)
    want = [f64(t) for t in grads]
    norm, _ = ob.clip(want, 1.0)
    got = float(g.GradClip(grads).clip(math.inf).double())
    assert abs(got - norm) <= norm * 20 * 2.0 ** -24


def test_mixed_magnitudes(lib):
    a, b = make([4000], [F32], scale=1e-25)[0], make([4000], [F32], seed=1, scale=1e-3)[0]
    z = torch.zeros(100_000, device="cuda")
    check([a, z, b], 1e-4, False)


def test_zero_gradients_and_empty_lists(lib):
    z = [torch.zeros(300, dtype=BF, device="cuda"), torch.zeros(5000, device="cuda")]
    plan = check(z, 1.0, False)
    assert float(plan.norm) == 0 and not plan.outs[0].any()
    for grads in ([], [torch.empty(0, device="cuda")], [torch.empty(0, device="cuda")] * 200):
        plan = g.GradClip(grads)
        plan.norm.fill_(3)
        assert float(plan.clip(1.0)) == 0


def test_tensors_then_empty_ones(lib):
    grads = make([50] * 96 + [0] * 10, [F32] * 106)
    check(grads, 0.01, False)
    grads = make([50] * 97 + [0] * 10, [F32] * 107)
    check(grads, 0.01, True)


def test_not_a_number_and_infinity(lib):
    grads = make([3000, 40], [BF, F32])
    grads[1][3] = float("nan")
    plan = g.GradClip(grads, [torch.zeros_like(t) for t in grads])
    assert math.isnan(float(plan.clip(1.0)))
    assert all(torch.isnan(o.float()).all() for o in plan.outs)
    grads[1][3] = float("inf")
    assert math.isinf(float(plan.clip(1.0)))
    o = plan.outs[1]
    assert torch.isnan(o[3]) and not torch.cat([o[:3], o[4:]]).any()


def test_same_bits_again_on_another_stream_and_in_a_graph(lib):
    grads = make([1_000_001, 4097, 300], [BF, F32, BF])
    outs = [torch.empty_like(t) for t in grads]
    plan = g.GradClip(grads, outs)
    n0 = plan.clip(0.5).clone()
    first = [o.clone() for o in outs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        n1 = plan.clip(0.5).clone()
    s.synchronize()
    assert torch.equal(n0, n1) and all(torch.equal(a, b) for a, b in zip(first, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.clip(0.5)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


def test_more_than_2_31_elements(lib):
    n = (1 << 31) + 12345
    t = torch.full((n,), 0.5, dtype=BF, device="cuda")
    t[-1] = 2.0
    out = torch.zeros_like(t)
    norm = float(g.GradClip([t], [out]).clip(1.0))
    want = math.sqrt(0.25 * (n - 1) + 4)
    assert abs(norm - want) <= want * 20 * 2.0 ** -24
    c = 1.0 / (want + 1e-6)
    for i in (0, 1 << 31, n - 2, n - 1):
        v = float(t[i]) * c
        assert abs(float(out[i]) - v) <= v * 2.0 ** -8
