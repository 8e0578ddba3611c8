"""The fp64 oracle of the step's operators: gradients against differences, the choice of experts
against an exhaustive one, and the 8-bit states' rounding."""
import numpy as np
import pytest

from oracle import step_ops as so


def differences(f, x, h=1e-6):
    """Central differences of a scalar function of an array."""
    d = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        lo, hi = x.copy(), x.copy()
        lo[i] -= h
        hi[i] += h
        d[i] = (f(hi) - f(lo)) / (2 * h)
    return d


def near(a, b):
    # a third derivative of order 1 times h^2 / 6, and roundings of f over 2 h
    assert np.abs(a - b).max() <= 1e-7 * max(1.0, np.abs(b).max())


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient(score, renorm):
    rng = np.random.default_rng(0)
    x, dw = rng.standard_normal((5, 7)), rng.standard_normal((5, 3))
    ids = np.array([[0, 1, 2], [6, 3, 3], [2, -1, 5], [-1, -1, -1], [4, 7, 4]])
    d, mag = so.route_grad(x, ids, dw, score, renorm, 2.5)
    near(d, differences(lambda a: (so.route_weights(a, ids, score, renorm, 2.5) * dw).sum(), x))
    assert (np.abs(d) <= mag * (1 + 1e-12)).all() and not d[3].any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("top", [1, 2])
def test_route_against_exhaustive_choice(score, bias, top):
    rng = np.random.default_rng(1)
    T, E, k, G, keep = 40, 12, 3, 4, 2
    x = np.round(rng.standard_normal((T, E)) * 4) / 4   # many ties
    b = np.round(rng.standard_normal(E)) / 4 if bias else None
    ids, w, _ = so.route(x, k, score, b, None, G, keep, top, True, 1.0)
    for t in range(T):
        s = so.sigmoid(x[t]) if score == "sigmoid" else so.softmax(x[t][None])[0]
        v = s if b is None else s + b
        c = x[t] if b is None else v
        group = [max(c[i:i + 3]) if top == 1 else sum(sorted(v[i:i + 3])[-2:])
                 for i in range(0, E, 3)]
        kept = sorted(range(G), key=lambda g: (-group[g], g))[:keep]
        want = sorted((e for e in range(E) if e // 3 in kept), key=lambda e: (-c[e], e))[:k]
        assert list(ids[t]) == want
        assert abs(w[t].sum() - 1) < 1e-12


@pytest.mark.parametrize("post,gate,branch,dh,dx", [
    (True, True, True, True, True), (False, True, True, True, True), (True, False, True, True, False),
    (False, False, False, True, True), (True, True, True, False, True)])
def test_residual_gradient(post, gate, branch, dh, dx):
    rng = np.random.default_rng(2)
    M, N, eps, scale = 3, 6, 1e-3, 0.7
    x, o, w, wp = (rng.standard_normal(s) for s in ((M, N), (M, N), N, N))
    gt = rng.standard_normal(M)
    gh, gx = rng.standard_normal((M, N)), rng.standard_normal((M, N))

    def loss(x=x, o=o, w=w, wp=wp, gt=gt):
        new = so.residual(x, o, wp, gt if gate else None, scale, post, eps) if branch else x
        return ((gh * so.normed(new, w, eps)).sum() if dh else 0.0) + ((gx * new).sum() if dx else 0)

    new = so.residual(x, o, wp, gt if gate else None, scale, post, eps) if branch else x
    d = so.residual_grad(gh if dh else None, gx if dx else None, new, o if branch else None,
                         wp if branch else None, gt if gate else None, w if dh else None, scale,
                         post, eps)
    near(d["dx"][0], differences(lambda a: loss(x=a), x))
    if dh:
        near(d["d_weight"][0], differences(lambda a: loss(w=a), w))
    if branch:
        near(d["do"][0], differences(lambda a: loss(o=a), o))
        near(d["d_post_weight"][0], differences(lambda a: loss(wp=a), wp))
        if gate:
            near(d["d_gate"][0], differences(lambda a: loss(gt=a), gt))


@pytest.mark.parametrize("signed", [True, False])
def test_held_values_keep_their_codes(signed):
    """A value that a code stands for is held by that code, whatever the random bits."""
    rng = np.random.default_rng(3)
    scales = np.array([32, 33, 90, 127, 200, 254], np.uint8)
    codes = rng.integers(0, 256, 6 * 256).astype(np.uint8)
    codes[::256] = 127 if signed else 255               # each block's largest, so that scales stay
    if signed:
        codes[codes == 128] = 0                         # -0 is held as 0
    x = so.decode(codes, scales, signed)
    for u in (0, 1, 65535):
        c, s = so.encode(x.astype(np.float32), np.full(len(x), u), signed)
        assert (c == codes).all() and (s == scales).all()


def test_rounding_is_fair():
    """Both neighbours are taken in proportion to the distance: the mean over all random bits is the
    value, to a sixteenth of 2^-16 of a step; below the least value to 2^-16 of it."""
    u = np.arange(65536)
    for signed, lowest in ((True, 2.0 ** -15 * 9 / 8), (False, 2.0 ** -31 * 9 / 8)):
        for v in (1.8, 1.3, 0.7531, 3.3e-3, lowest * 0.4, lowest * 1e-3):
            x = np.full(65536, v, np.float32)
            x[::256] = 1.875
            c, s = so.encode(x, u, signed)
            y = so.decode(c, s, signed)
            rest = np.arange(65536) % 256 != 0
            step = max(2.0 ** np.floor(np.log2(v)) / 8, lowest)
            # bits that are multiples of 256 are missing from the mean: at most one in 256 ups
            assert abs(y[rest].mean() - float(x[1])) <= step * (2.0 ** -8 + 2.0 ** -15)


def test_blocks_that_are_not_finite():
    x = np.ones(600, np.float32)
    x[300] = np.nan
    x[599] = np.inf
    c, s = so.encode(x, np.zeros(600, int), True)
    assert s[0] == 127 and (s[1:] == 255).all()
    assert np.isnan(so.decode(c, s, True)[256:]).all() and (so.decode(c, s, True)[:256] == 1).all()


def test_words_differ_between_tensors_and_steps():
    a = so.words(5, 1, 0, 4096)
    for b in (so.words(5, 1, 1, 4096), so.words(5, 2, 0, 4096), so.words(6, 1, 0, 4096),
              so.words(5 + (1 << 40), 1, 0, 4096), so.words(5, 1, 0, 4096, first=1 << 33)):
        assert (a == b).mean() < 0.01
    ones = [((a >> np.uint64(i)) & np.uint64(1)).mean() for i in range(32)]
    assert max(abs(np.array(ones) - 0.5)) < 5 * 0.5 / 64   # five standard deviations of 4096 bits


def test_adamw_against_a_scalar_loop():
    p, m, v = 0.3, 0.0, 0.0
    for t, g in enumerate((0.1, -0.2, 0.4), 1):
        p, m, v = so.adamw(p, g, m, v, t, 0.01, 0.9, 0.999, 1e-8, 0.1)
    q, m1, v1 = 0.3, 0.0, 0.0
    for t, g in enumerate((0.1, -0.2, 0.4), 1):
        m1 = 0.9 * m1 + 0.1 * g
        v1 = 0.999 * v1 + 0.001 * g * g
        q = q - 0.01 * 0.1 * q - 0.01 * (m1 / (1 - 0.9 ** t)) / ((v1 / (1 - 0.999 ** t)) ** 0.5
                                                                + 1e-8)
    assert abs(p - q) < 1e-15
