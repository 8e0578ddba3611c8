"""Block-128 E4M3 quantisers (bit-exact) and product against the fp64 oracle."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import block_ops as ob

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def up(n, m):
    return (n + m - 1) // m * m


def f32(t):
    return t.float().cpu().numpy()


def randbf(M, N, seed=0, scale=1.0, spread=False):
    gen = torch.Generator().manual_seed(seed * 65537 + M * 131 + N)
    x = torch.randn(M, N, generator=gen) * scale
    if spread:  # rows and columns of very different size, zeros, a row of zeros
        x *= 2.0 ** torch.randint(-20, 20, (M, 1), generator=gen)
        x *= 2.0 ** torch.randint(-3, 3, (1, N), generator=gen)
        x[torch.rand(M, N, generator=gen) < 0.05] = 0
        x[M // 2] = 0
    return x.to(BF).cuda()


def quant_rows(x, row=True, col=True, pad=0, vec=True):
    M, N = x.shape
    m = 16 if vec else 1
    qr = torch.full((M, up(N, m) + pad), 0x55, dtype=torch.uint8, device="cuda")
    sr = torch.full((-(-N // 128), up(M, 4) + pad), 7.0, device="cuda")
    qc = torch.full((N, up(M, m) + pad), 0x55, dtype=torch.uint8, device="cuda")
    sc = torch.full((-(-M // 128), up(N, 4) + pad), 7.0, device="cuda")
    kw = {}
    if row:
        kw.update(q_row=qr, ld_qrow=qr.shape[1], s_row=sr, ld_srow=sr.shape[1])
    if col:
        kw.update(q_col=qc, ld_qcol=qc.shape[1], s_col=sc, ld_scol=sc.shape[1])
    g.fp8_block_quantize_rows(x, x.stride(0), M, N, **kw)
    return qr, sr, qc, sc


def check_rows(x, out, row=True, col=True):
    qr, sr, qc, sc = out
    M, N = x.shape
    X = f32(x)
    for on, q, s, ref, w in ((row, qr, sr, X, N), (col, qc, sc, np.ascontiguousarray(X.T), M)):
        if not on:
            assert (q == 0x55).all() and (s == 7.0).all()
            continue
        eq, es = ob.quantize_rows(ref)
        np.testing.assert_array_equal(ob.e4m3_values(q[:, :w].cpu().numpy()), eq)
        np.testing.assert_array_equal(s[:, :ref.shape[0]].cpu().numpy(), es)
        assert (q[:, w:] == 0x55).all() and (s[:, ref.shape[0]:] == 7.0).all()


@pytest.mark.parametrize("M,N", [(1, 1), (1, 128), (3, 7), (1, 7168), (16, 130), (127, 129),
                                 (128, 128), (129, 256), (257, 1000), (300, 2880), (1000, 333)])
def test_quantize_rows(lib, M, N):
    for spread in (False, True):
        x = randbf(M, N, spread=spread)
        check_rows(x, quant_rows(x))
        check_rows(x, quant_rows(x, col=False), col=False)
        check_rows(x, quant_rows(x, row=False), row=False)


def test_quantize_rows_strides(lib):
    x = torch.zeros(70, 300, dtype=BF, device="cuda")
    for w, off in ((256, 8), (255, 0), (200, 3)):
        v = x[:, off:off + w]
        v.copy_(randbf(70, w))
        check_rows(v, quant_rows(v, pad=16))
        check_rows(v, quant_rows(v, pad=3, vec=False))


@pytest.mark.parametrize("N,K", [(1, 1), (5, 128), (128, 130), (129, 127), (256, 384), (300, 1001),
                                 (2880, 720)])
def test_quantize_weight(lib, N, K):
    w = randbf(N, K, scale=0.02, spread=True)
    nb, kb = -(-N // 128), -(-K // 128)
    q = torch.full((N, up(K, 16)), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.zeros(nb, kb, device="cuda")
    qt = torch.full((K, up(N, 16)), 0x55, dtype=torch.uint8, device="cuda")
    st = torch.zeros(kb, nb, device="cuda")
    g.fp8_block_quantize_weight(w, K, N, K, q, q.shape[1], s, qt, qt.shape[1], st)
    eq, es = ob.quantize_weight(f32(w))
    np.testing.assert_array_equal(s.cpu().numpy(), es)
    np.testing.assert_array_equal(st.cpu().numpy(), es.T)
    np.testing.assert_array_equal(ob.e4m3_values(q[:, :K].cpu().numpy()), eq)
    assert torch.equal(qt[:, :N], q[:, :K].t())
    q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
    g.fp8_block_quantize_weight(w, K, N, K, q2, q.shape[1], s2)
    assert torch.equal(q2[:, :K], q[:, :K]) and torch.equal(s2, s)


def test_quantize_not_a_number_and_infinity(lib):
    x = randbf(4, 256)
    x[0, 3] = float("nan")
    x[1, 200] = float("inf")
    q, s, _, _ = quant_rows(x, col=False)
    v = ob.e4m3_values(q.cpu().numpy()) * np.repeat(s[:, :4].cpu().numpy(), 128, 0).T
    bad = np.isnan(v)
    assert bad[0].sum() == 1 and bad[0, 3]
    assert not bad[1, :128].any() and bad[1, 128:].all() and not bad[2:].any()


def rand_codes(rows, cols, seed, ld=None):
    """E4M3 codes of every magnitude but NaN; the bytes past a row's end are NaN codes."""
    r = np.random.default_rng([seed, rows, cols])
    c = r.integers(0, 256, (rows, cols)).astype(np.uint8)
    c[(c & 127) == 127] = 0x30
    full = np.full((rows, ld or up(cols, 16)), 0x7F, np.uint8)
    full[:, :cols] = c
    return torch.from_numpy(full).cuda(), ob.e4m3_values(c)


def rand_scales(a, b, seed, ld=None):
    r = np.random.default_rng([seed, a, b, 1])
    s = (2.0 ** r.uniform(-3, 3, (a, b))).astype(np.float32)
    full = np.full((a, ld or b), np.nan, np.float32)
    full[:, :b] = s
    return torch.from_numpy(full).cuda(), s


def check_gemm(M, N, K, block, dt=BF, ldc=None, seed=0, c_off=0):
    kb = -(-K // 128)
    a, av = rand_codes(M, K, seed)
    b, bv = rand_codes(N, K, seed + 1, up(K, 16) + 16)
    sa, sav = rand_scales(kb, M, seed, up(M, 4))
    if block:
        sb, sbv = rand_scales(-(-N // 128), kb, seed + 1)
        B = ob.blocks_scaled(bv, sbv)
    else:
        sb, sbv = rand_scales(kb, N, seed + 1, up(N, 4) + 4)
        B = ob.rows_scaled(bv, sbv)
    A = ob.rows_scaled(av, sav)
    ldc = ldc or N
    buf = torch.full((M * ldc + c_off + 8,), 7.0, dtype=dt, device="cuda")
    c = buf[c_off:c_off + M * ldc].view(M, ldc)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    g.fp8_block_gemm(a, a.shape[1], sa, sa.shape[1], b, b.shape[1], sb, sb.shape[1], int(block), c,
                     ldc, 0 if dt == BF else 1, M, N, K, err)
    torch.cuda.synchronize()
    assert int(err) == 0
    want, size = A @ B.T, np.abs(A) @ np.abs(B).T
    # a k-block's 128 products are added with at least 20 bits below the largest of them, the
    # k-blocks in fp32; then the result's own rounding
    half = 2.0 ** -8 if dt == BF else 2.0 ** -24
    tol = half * 1.01 * np.abs(want) + 2.0 ** -15 * size
    got = c[:, :N].double().cpu().numpy()
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4].tolist())
    assert (c[:, N:] == 7).all() and (buf[:c_off] == 7).all() and (buf[c_off + M * ldc:] == 7).all()


MS = [1, 2, 7, 16, 17, 33, 64, 65, 128, 129, 200, 256, 300]


@pytest.mark.parametrize("M", MS)
@pytest.mark.parametrize("block", [True, False])
def test_gemm_row_counts(lib, M, block):
    for N, K in ((1, 128), (129, 300), (256, 1024)):
        check_gemm(M, N, K, block)


@pytest.mark.parametrize("N", [1, 2, 8, 31, 64, 100, 128, 255, 257, 384, 1000])
@pytest.mark.parametrize("block", [True, False])
def test_gemm_column_counts(lib, N, block):
    for M, K in ((3, 200), (130, 272), (520, 640)):
        check_gemm(M, N, K, block)


@pytest.mark.parametrize("K", [1, 15, 16, 31, 32, 33, 64, 100, 127, 128, 129, 160, 256, 257, 1000,
                               2048, 2880, 7168])
@pytest.mark.parametrize("block", [True, False])
def test_gemm_lengths(lib, K, block):
    check_gemm(20, 136, K, block)
    check_gemm(140, 264, K, block)


@pytest.mark.parametrize("block", [True, False])
def test_gemm_outputs(lib, block):
    for M, N, K in ((40, 200, 512), (300, 520, 512)):
        check_gemm(M, N, K, block, dt=F32)
        check_gemm(M, N, K, block, ldc=N + 8)
        check_gemm(M, N, K, block, ldc=N + 3)
        check_gemm(M, N, K, block, c_off=1)
        check_gemm(M, N, K, block, dt=F32, ldc=N + 1, c_off=1)


@pytest.mark.parametrize("M,N,K", [(700, 900, 1100), (1999, 1440, 1440), (2049, 2300, 600)])
@pytest.mark.parametrize("block", [True, False])
def test_gemm_many_tiles(lib, M, N, K, block):
    check_gemm(M, N, K, block)


def test_nan_codes_reach_only_their_row_and_column(lib):
    M, N, K = 40, 300, 400
    x, w = randbf(M, K), randbf(N, K, scale=0.02, seed=2)
    x[7, 350] = float("nan")
    w[250, 20] = float("inf")
    lin = g.Fp8Linear(N, K, M, train=False)
    lin.set_weight(w)
    y = torch.isnan(lin.forward(x).float()).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[7] = True
    want[:, 128:256] = True  # the infinite scale poisons its block's 128 features
    np.testing.assert_array_equal(y, want)


def linear_oracle(x, w, dy):
    X, W, D = f32(x), f32(w), f32(dy)
    xq = ob.rows_scaled(*ob.quantize_rows(X))
    wq = ob.blocks_scaled(*ob.quantize_weight(W))
    dq = ob.rows_scaled(*ob.quantize_rows(D))
    xt = ob.rows_scaled(*ob.quantize_rows(np.ascontiguousarray(X.T)))
    dt = ob.rows_scaled(*ob.quantize_rows(np.ascontiguousarray(D.T)))
    return [(a @ b, np.abs(a) @ np.abs(b)) for a, b in ((xq, wq.T), (dq, wq), (dt, xt.T))]


@pytest.mark.parametrize("M,N,K", [(1, 64, 64), (5, 100, 130), (64, 256, 128), (129, 130, 257),
                                   (333, 720, 1440)])
def test_linear_training_step(lib, M, N, K):
    x, w, dy = randbf(M, K), randbf(N, K, scale=0.02, seed=1), randbf(M, N, scale=0.1, seed=2)
    lin = g.Fp8Linear(N, K, M + 9)
    lin.set_weight(w)
    y = lin.forward(x)
    dx, dw = lin.backward(dy)
    torch.cuda.synchronize()
    assert int(lin.err) == 0
    for got, (want, size) in zip((y, dx, dw), linear_oracle(x, w, dy)):
        err = np.abs(got.double().cpu().numpy() - want)
        assert (err <= 2.0 ** -8 * 1.01 * np.abs(want) + 2.0 ** -15 * size).all()


def test_linear_gradients_against_differences(lib):
    """The layer is linear in each argument up to quantisation: with values that E4M3 holds
    exactly (small integers under a power-of-two scale, each block's maximum 448) the difference
    of two forward passes is the gradient times the step, up to the outputs' bf16 rounding."""
    r = np.random.default_rng(0)
    M, N, K = 128, 128, 128
    vals = np.array([-448.0, -16, -8, -4, -2, -1, 0, 1, 2, 4, 8, 16, 448])

    def exact(rows, cols):
        v = r.choice(vals[1:-1], (rows, cols))
        i = np.arange(128)
        v[i, (5 * i + 3) % 128] = 448.0      # one in every row and every column
        return torch.from_numpy(v).to(BF).cuda()

    x, w, dy = exact(M, K), exact(N, K), exact(M, N)
    lin = g.Fp8Linear(N, K, M)
    lin.set_weight(w)
    lin.forward(x)
    dx, dw = (t.double().cpu().numpy() for t in lin.backward(dy))
    D = dy.double().cpu().numpy()

    def value(x, w):
        lin.set_weight(w)
        y = lin.forward(x).double().cpu().numpy()
        return (y * D).sum(), (np.abs(y) * np.abs(D)).sum() * 2.0 ** -8

    v0, e0 = value(x, w)
    for arg, grad in ((x, dx), (w, dw)):
        for _ in range(6):
            i, j = int(r.integers(128)), int(r.integers(128))
            if float(arg[i, j]) == 448.0:
                continue
            keep = float(arg[i, j])
            arg[i, j] = keep + (16 if keep <= 0 else -16)  # exact: no new block maximum
            step = float(arg[i, j]) - keep
            if float(arg[i, j]) not in vals:
                arg[i, j] = 0.0
                step = -keep
            v1, e1 = value(x, w)
            arg[i, j] = keep
            assert abs((v1 - v0) - step * grad[i, j]) <= e0 + e1 + abs(step * grad[i, j]) * 2.0 ** -8


def test_no_rows(lib):
    lin = g.Fp8Linear(64, 64, 8)
    lin.set_weight(randbf(64, 64))
    assert lin.forward(torch.empty(0, 64, dtype=BF, device="cuda")).shape == (0, 64)
    dx, dw = lin.backward(torch.empty(0, 64, dtype=BF, device="cuda"))
    assert dx.shape == (0, 64) and not dw.any()


def test_same_bits_again_on_another_stream_and_in_a_graph(lib):
    for M, N, K in ((1, 512, 1024), (48, 512, 2048), (700, 640, 512)):
        x, w, dy = randbf(M, K), randbf(N, K, scale=0.02, seed=1), randbf(M, N, seed=2)
        lin = g.Fp8Linear(N, K, M)

        def once():
            lin.set_weight(w)
            y = lin.forward(x)
            return [t.clone() for t in (y, *lin.backward(dy))]

        first = once()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            other = once()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            lin.set_weight(w)
            y = lin.forward(x)
            dx, dw = lin.backward(dy)
        for t in (y, dx, dw):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(first, other, (y, dx, dw)):
            assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("pad,off", [(0, 0), (0, 1), (1, 0), (2, 3), (3, 5), (5, 6), (7, 7)])
@pytest.mark.parametrize("block", [True, False])
def test_gemm_rows_off_boundaries(lib, block, pad, off):
    """Whole tiles whose rows start anywhere in a 16-byte block, and the last, partial ones."""
    check_gemm(2500, 2301, 130, block, ldc=2301 + pad, c_off=off)
    check_gemm(1300, 135, 300, block, ldc=135 + pad, c_off=off)


@pytest.mark.parametrize("off", range(8))
def test_quantize_rows_off_boundaries(lib, off):
    for M, N, ld in ((130, 257, 257), (70, 1000, 1003), (9, 130, 131), (300, 127, 129)):
        buf = randbf(1, M * ld + 16, seed=off)[0]
        x = buf[off:off + M * ld].view(M, ld)[:, :N]
        check_rows(x, quant_rows(x))
        check_rows(x, quant_rows(x, col=False), col=False)
