"""Pins of the fp64 oracle of the operators around the expert layer: gradients against central
differences, the E4M3 rounding against an exhaustive search, and simple known values."""
import numpy as np
import pytest

from oracle import block_ops as ob


def test_router_loss_of_a_uniform_router_is_its_coefficient():
    T, E, k = 24, 6, 2
    ids = np.stack([np.arange(T) % E, (np.arange(T) + 1) % E], axis=1)
    loss, counts, mean_prob, f, n = ob.router_loss(np.zeros((T, E)), ids, 0.01)
    assert n == T and (counts == T * k // E).all()
    np.testing.assert_allclose(mean_prob, 1 / E)
    np.testing.assert_allclose(f, 1.0)
    assert loss == pytest.approx(0.01, rel=1e-12)


def test_router_gradient_matches_differences():
    r = np.random.default_rng(0)
    T, E, k = 5, 7, 3
    x = r.standard_normal((T, E))
    ids = np.argsort(-x, axis=1)[:, :k]
    mask = np.array([1, 1, 0, 1, 1])
    g = r.standard_normal((T, k))
    h = 1e-6

    def value(z):
        loss, *_ = ob.router_loss(z, ids, 0.3, mask)
        c = np.take_along_axis(z, ids, axis=1)
        w = np.exp(c) / np.exp(c).sum(axis=1, keepdims=True)
        return 1.7 * loss + (w * g).sum()

    c = np.take_along_axis(x, ids, axis=1)
    w = np.exp(c) / np.exp(c).sum(axis=1, keepdims=True)
    d, _ = ob.router_grad(x, ids, 0.3, mask, 1.7, w, g)
    for t in range(T):
        for e in range(E):
            z = x.copy()
            z[t, e] += h
            up = value(z)
            z[t, e] -= 2 * h
            assert d[t, e] == pytest.approx((up - value(z)) / (2 * h), rel=1e-5, abs=1e-8)


def test_layernorm_gradient_matches_differences():
    r = np.random.default_rng(1)
    M, N, eps, h = 3, 9, 1e-5, 1e-6
    x, dy = r.standard_normal((M, N)), r.standard_normal((M, N))
    gamma, beta = r.standard_normal(N), r.standard_normal(N)

    def value(x, gamma, beta):
        return float((ob.layernorm(x, gamma, beta, eps)[0] * dy).sum())

    _, mean, rstd = ob.layernorm(x, gamma, beta, eps)
    dx, dg, db, _, _ = ob.layernorm_grad(dy, x, gamma, mean, rstd)
    for arr, grad in ((x, dx), (gamma, dg), (beta, db)):
        for i in np.ndindex(arr.shape):
            keep = arr[i]
            arr[i] = keep + h
            up = value(x, gamma, beta)
            arr[i] = keep - h
            down = value(x, gamma, beta)
            arr[i] = keep
            assert grad[i] == pytest.approx((up - down) / (2 * h), rel=1e-5, abs=1e-7)


def test_e4m3_rounding_against_all_codes():
    codes = np.arange(256, dtype=np.uint8)
    vals = ob.e4m3_values(codes)
    fin = np.unique(vals[np.isfinite(vals)])
    assert fin.max() == 448.0 and fin[fin > 0].min() == 2.0 ** -9
    r = np.random.default_rng(2)
    v = np.concatenate([r.standard_normal(2000) * 2.0 ** r.integers(-12, 9, 2000),
                        (fin[1:] + fin[:-1]) / 2, fin, [449.0, 1e9, -1e9]])
    got = ob.e4m3_nearest(v)
    man = {x: int(c) & 1 for c, x in zip(codes, vals) if np.isfinite(x)}
    for a, b in zip(v, got):
        d = np.abs(fin - a)
        best = fin[d == d.min()]
        want = best[0] if len(best) == 1 else [x for x in best if man[x] == 0][0]
        assert b == want, (a, b, want)


def test_block_scales():
    x = np.zeros((2, 200), np.float32)
    x[0, 5], x[0, 150], x[1, 199] = -896.0, 2.0, 1e-3
    q, s = ob.quantize_rows(x)
    tiny = np.float32(2.0 ** -100) / np.float32(448)
    assert s.shape == (2, 2) and s[0, 0] == 2.0 and s[0, 1] == tiny
    assert s[1, 0] == np.float32(2.0) / np.float32(448)
    assert q[0, 5] == -448 and q[0, 150] == 448 and not q[1, :128].any()
    v = ob.rows_scaled(q, s)
    np.testing.assert_allclose(v, x, rtol=2.0 ** -4)
