"""Layer norm forward and backward against the fp64 oracle and against differences."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import block_ops as ob

pytestmark = pytest.mark.gpu
ULP = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (BF, F32), (F32, F32)]
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}  # half an ulp of a result, relative


def f64(t):
    return t.detach().double().cpu().numpy()


def make(M, N, xt, wt, seed=0, mean=0.5, scale=1.0):
    gen = torch.Generator().manual_seed(seed * 7919 + M * 31 + N)
    x = (torch.randn(M, N, generator=gen) * scale + mean).to(xt).cuda()
    dy = torch.randn(M, N, generator=gen).to(xt).cuda()
    gamma = (1 + 0.2 * torch.randn(N, generator=gen)).to(wt).cuda()
    beta = (0.3 * torch.randn(N, generator=gen)).to(wt).cuda()
    return x, dy, gamma, beta


def check_fwd(x, gamma, beta, out, eps):
    y, mean, rstd = out
    N = x.shape[1]
    X = f64(x)
    ey, em, er = ob.layernorm(X, None if gamma is None else f64(gamma),
                              None if beta is None else f64(beta), eps)
    # fp32 sums of N terms: at most N/1024 + 64 additions in a row, each 1 ulp of the partial sum
    c = (64 + N / 512) * ULP
    absmean = np.abs(X).mean(axis=1)
    assert (np.abs(f64(mean) - em) <= c * absmean + 1e-44).all()
    # the mean's error moves x - mean; squared it is a second-order term of the variance
    sens = c * (2 + absmean * er)
    assert (np.abs(f64(rstd) - er) <= er * sens).all()
    h = np.abs((X - em[:, None]) * er[:, None])
    gm = 1.0 if gamma is None else np.abs(f64(gamma))
    tol = HALF[y.dtype] * 1.01 * np.abs(ey) + gm * (sens[:, None] * (1 + h)) + \
        4 * ULP * (gm * h + (0 if beta is None else np.abs(f64(beta))))
    assert (np.abs(f64(y) - ey) <= tol + 1e-40).all()


def check_bwd(dy, x, gamma, mean, rstd, out):
    dx, dg, db = out
    X, DY = f64(x), f64(dy)
    G = None if gamma is None else f64(gamma)
    mu, rs = f64(mean), f64(rstd)
    M, N = X.shape
    ex, eg, eb, sg, sb = ob.layernorm_grad(DY, X, G, mu, rs)
    h = np.abs((X - mu[:, None]) * rs[:, None])
    hh = h + 1.0
    u = np.abs(DY * (1.0 if G is None else G))
    c = (64 + N / 512) * ULP
    terms = rs[:, None] * (u + u.mean(axis=1, keepdims=True)
                           + h * (u * hh).mean(axis=1, keepdims=True))
    assert (np.abs(f64(dx) - ex) <= HALF[dx.dtype] * 1.01 * np.abs(ex) + c * terms + 1e-40).all()
    # columns: at most M/32 + 64 additions in a row
    cc = (64 + M / 32) * ULP
    if dg is not None:
        assert (np.abs(f64(dg) - eg) <= HALF[dg.dtype] * 1.01 * np.abs(eg) + cc * (sg + sb)
                + 1e-40).all()
    if db is not None:
        assert (np.abs(f64(db) - eb) <= HALF[db.dtype] * 1.01 * np.abs(eb) + cc * sb
                + 1e-40).all()


SIZES = [1, 2, 7, 8, 31, 33, 64, 100, 128, 250, 256, 257, 512, 520, 1000, 1024, 1032, 2047, 2048,
         2880, 4095, 4096, 4104, 7168, 8192, 9000, 9001, 16384, 16390, 20000]


@pytest.mark.parametrize("N", SIZES)
@pytest.mark.parametrize("xt,wt", TYPES)
def test_matches_oracle(lib, N, xt, wt):
    for M in (1, 5, 67):
        x, dy, gamma, beta = make(M, N, xt, wt)
        ln = g.LayerNorm(N, M, dtype=xt, weight_dtype=wt, eps=1e-5)
        out = ln.forward(x, gamma, beta)
        check_fwd(x, gamma, beta, out, 1e-5)
        check_bwd(dy, x, gamma, out[1], out[2], ln.backward(dy, x, gamma))


@pytest.mark.parametrize("M,N,xt,wt", [(3000, 96, BF, BF), (1999, 2880, BF, F32),
                                       (700, 1001, F32, F32), (40000, 33, BF, F32)])
def test_many_rows(lib, M, N, xt, wt):
    x, dy, gamma, beta = make(M, N, xt, wt, seed=3)
    ln = g.LayerNorm(N, M, dtype=xt, weight_dtype=wt)
    out = ln.forward(x, gamma, beta)
    check_fwd(x, gamma, beta, out, 1e-5)
    check_bwd(dy, x, gamma, out[1], out[2], ln.backward(dy, x, gamma))


@pytest.mark.parametrize("N", [64, 100, 4096, 20000])
def test_no_weights(lib, N):
    x, dy, gamma, beta = make(9, N, BF, BF)
    ln = g.LayerNorm(N, 9)
    out = ln.forward(x)
    check_fwd(x, None, None, out, 1e-5)
    check_bwd(dy, x, None, out[1], out[2], ln.backward(dy, x))
    check_fwd(x, gamma, None, ln.forward(x, gamma), 1e-5)
    check_fwd(x, None, beta, ln.forward(x, None, beta), 1e-5)


@pytest.mark.parametrize("pad,shift", [(8, 0), (3, 0), (8, 1), (8, 4)])
@pytest.mark.parametrize("xt", [BF, F32])
def test_row_strides_and_offsets(lib, pad, shift, xt):
    M, N = 37, 264
    x0, dy0, gamma, beta = make(M, N, xt, xt)

    def strided(t):
        buf = torch.full((M * (N + pad) + 8,), float("nan"), dtype=xt, device="cuda")
        v = buf[shift:shift + M * (N + pad)].view(M, N + pad)[:, :N]
        v.copy_(t)
        return v

    x, dy = strided(x0), strided(dy0)
    wg = strided(gamma.expand(M, N))[0]   # weights off 16-byte boundaries too
    ln = g.LayerNorm(N, M, dtype=xt)
    out = ln.forward(x, wg, beta)
    check_fwd(x0, gamma, beta, out, 1e-5)
    check_bwd(dy0, x0, gamma, out[1], out[2], ln.backward(dy, x, wg))


@pytest.mark.parametrize("N", [72, 3001, 20000])
def test_in_place(lib, N):
    M = 11
    x, dy, gamma, beta = make(M, N, BF, BF)
    ln = g.LayerNorm(N, M)
    y, mean, rstd = ln.forward(x, gamma, beta)
    dx, dg, db = (t.clone() for t in ln.backward(dy, x, gamma))
    x2 = x.clone()
    g.moe_layernorm_fwd(x2, N, gamma, beta, x2, N, None, None, M, N, 1e-5, 0, 0)
    assert torch.equal(x2, y)
    for target in ("dy", "x"):
        a, b = dy.clone(), x.clone()
        dst = a if target == "dy" else b
        g.moe_layernorm_bwd(a, N, b, N, gamma, mean, rstd, dst, N, ln.dgamma, ln.dbeta, M, N, 0, 0,
                            ln.ws, ln.ws_bytes)
        assert torch.equal(dst, dx) and torch.equal(ln.dgamma, dg) and torch.equal(ln.dbeta, db)


def test_large_mean_constant_rows_and_zero_eps(lib):
    # a mean a thousand times the spread; a row without spread has y = beta
    M, N = 8, 1000
    x, dy, gamma, beta = make(M, N, F32, F32, mean=1000.0)
    x[3] = 5.0
    ln = g.LayerNorm(N, M, dtype=F32)
    out = ln.forward(x, gamma, beta)
    check_fwd(x, gamma, beta, out, 1e-5)
    assert torch.equal(out[0][3], beta)
    check_bwd(dy, x, gamma, out[1], out[2], ln.backward(dy, x, gamma))


def test_not_a_number_stays_in_its_row(lib):
    x, dy, gamma, beta = make(6, 512, BF, BF)
    x[2, 17] = float("nan")
    x[4, 3] = float("inf")
    ln = g.LayerNorm(512, 6)
    y, mean, rstd = ln.forward(x, gamma, beta)
    bad = torch.isnan(y.float()).any(dim=1).cpu().tolist()
    assert bad == [False, False, True, False, True, False]


def test_partial_gradients_and_no_rows(lib):
    x, dy, gamma, beta = make(20, 96, BF, BF)
    ln = g.LayerNorm(96, 20)
    _, mean, rstd = ln.forward(x, gamma, beta)
    dx, dg, db = (t.clone() for t in ln.backward(dy, x, gamma))
    only = torch.empty_like(dg)
    g.moe_layernorm_bwd(dy, 96, x, 96, gamma, mean, rstd, ln.dx, 96, only, None, 20, 96, 0, 0,
                        ln.ws, ln.ws_bytes)
    assert torch.equal(only, dg)
    out = torch.empty_like(x)
    g.moe_layernorm_bwd(dy, 96, x, 96, gamma, mean, rstd, out, 96, None, None, 20, 96, 0, 0, None,
                        0)
    assert torch.equal(out, dx)
    only.fill_(3)
    g.moe_layernorm_bwd(None, 96, None, 96, None, None, None, None, 96, only, db, 0, 96, 0, 0,
                        ln.ws, ln.ws_bytes)
    assert not only.any() and not db.any()
    assert ln.forward(x[:0], gamma, beta)[0].shape == (0, 96)


def test_gradient_against_differences(lib):
    """fp32 kernels; the loss sum(y * dy) in fp64 from fp32 y. Step 2^-5: truncation h^2/6 times
    third derivatives (below 8 for unit rows), rounding 2 * N * ulp / h."""
    M, N, h = 2, 12, 2.0 ** -5
    x, dy, gamma, beta = make(M, N, F32, F32)
    ln = g.LayerNorm(N, M, dtype=F32)
    ln.forward(x, gamma, beta)
    dx, dg, db = (f64(t) for t in ln.backward(dy, x, gamma))
    D = f64(dy)

    def value():
        return float((f64(ln.forward(x, gamma, beta)[0]) * D).sum())

    scale = float(np.abs(D).max()) * 2
    tol = scale * (8 * h * h / 6 * 4 + 2 * N * ULP * 4 / h)
    for t, grad in ((x, dx), (gamma, dg), (beta, db)):
        flat, gf = t.view(-1), grad.reshape(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + h
            up = value()
            flat[i] = keep - h
            down = value()
            flat[i] = keep
            assert abs((up - down) / (2 * h) - gf[i]) <= tol


def test_same_bits_again_on_another_stream_and_in_a_graph(lib):
    x, dy, gamma, beta = make(3000, 1024, BF, BF)
    ln = g.LayerNorm(1024, 3000)

    def once():
        out = ln.forward(x, gamma, beta)
        return [t.clone() for t in (*out, *ln.backward(dy, x, gamma))]

    first = once()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        other = once()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, mean, rstd = ln.forward(x, gamma, beta)
        dx, dg, db = ln.backward(dy, x, gamma)
    for t in (y, mean, rstd, dx, dg, db):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b, c in zip(first, other, (y, mean, rstd, dx, dg, db)):
        assert torch.equal(a, b) and torch.equal(a, c)


OFF = [(2500, 1), (2500, 7), (2500, 63), (2500, 130), (2500, 249), (2500, 250), (2500, 257),
       (1300, 333), (1300, 505), (1300, 511), (700, 1017), (700, 1018), (700, 1025), (700, 2041),
       (700, 2047), (400, 3065), (400, 3071), (400, 4089), (400, 5113), (400, 5121), (320, 8185),
       (320, 10233), (320, 10241), (320, 16377), (320, 16383)]


@pytest.mark.parametrize("M,N", OFF)
@pytest.mark.parametrize("xt,wt", TYPES)
def test_many_rows_off_boundaries(lib, M, N, xt, wt):
    x, dy, gamma, beta = make(M, N, xt, wt, seed=5)
    ln = g.LayerNorm(N, M, dtype=xt, weight_dtype=wt)
    out = ln.forward(x, gamma, beta)
    check_fwd(x, gamma, beta, out, 1e-5)
    check_bwd(dy, x, gamma, out[1], out[2], ln.backward(dy, x, gamma))


@pytest.mark.parametrize("shift", [0, 1, 3, 6])
@pytest.mark.parametrize("M,N,pad", [(33, 301, 2), (700, 61, 1), (700, 301, 3), (700, 1003, 5),
                                     (400, 2200, 9), (330, 4097, 2), (320, 9000, 1)])
@pytest.mark.parametrize("xt", [BF, F32])
def test_rows_beside_not_a_number(lib, M, N, pad, shift, xt):
    """Rows that share 16-byte blocks with NaNs: none gets in, and none is overwritten."""
    x0, dy0, gamma0, beta0 = make(M, N, xt, xt, seed=6)
    ld = N + pad

    def strided(t=None):
        buf = torch.full((M * ld + 16,), float("nan"), dtype=xt, device="cuda")
        v = buf[shift:shift + M * ld].view(M, ld)[:, :N]
        if t is not None:
            v.copy_(t)
        return buf, v

    def weight(t):  # off 16-byte boundaries, NaNs around it
        buf = torch.full((N + 16,), float("nan"), dtype=xt, device="cuda")
        buf[shift:shift + N] = t
        return buf[shift:shift + N]

    code = 0 if xt is BF else 1
    (_, x), (_, dy), (yb, y), (dxb, dx) = strided(x0), strided(dy0), strided(), strided()
    gamma, beta = weight(gamma0), weight(beta0)
    mean = torch.empty(M, device="cuda")
    rstd = torch.empty(M, device="cuda")
    dg, db = torch.empty(N, dtype=xt, device="cuda"), torch.empty(N, dtype=xt, device="cuda")
    n = g.moe_layernorm_workspace(M, N)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    g.moe_layernorm_fwd(x, ld, gamma, beta, y, ld, mean, rstd, M, N, 1e-5, code, code)
    check_fwd(x0, gamma0, beta0, (y, mean, rstd), 1e-5)
    g.moe_layernorm_bwd(dy, ld, x, ld, gamma, mean, rstd, dx, ld, dg, db, M, N, code, code, ws, n)
    check_bwd(dy0, x0, gamma0, mean, rstd, (dx, dg, db))
    for buf, v in ((yb, y), (dxb, dx)):
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[shift:shift + M * ld].view(M, ld)[:, :N] = False
        assert torch.isnan(buf[keep]).all()
    want = dx.clone()
    g.moe_layernorm_bwd(dy, ld, x, ld, gamma, mean, rstd, dy, ld, dg, db, M, N, code, code, ws, n)
    assert torch.equal(dy, want)  # in place
    want = y.clone()
    g.moe_layernorm_fwd(x, ld, gamma, beta, x, ld, mean, rstd, M, N, 1e-5, code, code)
    assert torch.equal(x, want)
