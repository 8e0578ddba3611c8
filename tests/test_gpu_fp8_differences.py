"""The FP8 layer's gradients against differences of products that are exact, so that a wrong
gradient cannot hide in the outputs' rounding."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
SIZE = 128
VALUES = np.array([-16.0, -8, -4, -2, -1, 0, 1, 2, 4, 8, 16])  # E4M3 holds them under a scale of 1


def exact(r):
    """Every row and every column has its largest value, 448, so that all scales are 1."""
    v = r.choice(VALUES, (SIZE, SIZE))
    i = np.arange(SIZE)
    v[i, (5 * i + 3) % SIZE] = 448.0
    return torch.from_numpy(v).to(BF).cuda()


def product(x, w):
    """x w^T in fp32 through the layer's own quantisers and product: integers below 2^24, a sum's
    terms within 2^18 of each other, so nothing is rounded."""
    n = SIZE
    q, s = torch.empty(n, n, dtype=torch.uint8).cuda(), torch.empty(1, n).cuda()
    wq, ws = torch.empty(n, n, dtype=torch.uint8).cuda(), torch.empty(1, 1).cuda()
    y = torch.empty(n, n).cuda()
    g.fp8_block_quantize_rows(x, n, n, n, q_row=q, ld_qrow=n, s_row=s, ld_srow=n)
    g.fp8_block_quantize_weight(w, n, n, n, wq, n, ws)
    g.fp8_block_gemm(q, n, s, n, wq, n, ws, 1, 1, y, n, g.DTYPE["fp32"], n, n, n)
    return y.double().cpu().numpy()


def test_gradients_are_the_differences_of_exact_products(lib):
    r = np.random.default_rng(0)
    x, w, dy = exact(r), exact(r), exact(r)
    lin = g.Fp8Linear(SIZE, SIZE, SIZE)
    lin.set_weight(w)
    lin.forward(x)
    dx, dw = (t.double().cpu().numpy() for t in lin.backward(dy))
    D = dy.double().cpu().numpy()
    y0 = product(x, w)
    X, W = x.double().cpu().numpy(), w.double().cpu().numpy()
    assert (y0 == X @ W.T).all()
    seen = told_apart = 0
    for arg, grad in ((x, dx), (w, dw)):
        for _ in range(40):
            i, j = int(r.integers(SIZE)), int(r.integers(SIZE))
            keep = float(arg[i, j])
            if keep == 448.0:
                continue
            step = float(r.choice(VALUES[VALUES != keep])) - keep
            arg[i, j] = keep + step
            change = float(((product(x, w) - y0) * D).sum()) / step
            arg[i, j] = keep
            tol = 2.0 ** -8 * abs(change)  # the gradient's own rounding to bf16
            assert abs(grad[i, j] - change) <= tol, (i, j, grad[i, j], change)
            seen += 1
            told_apart += abs(0.0 - change) > tol and abs(-grad[i, j] - change) > tol
    assert seen >= 60 and told_apart >= seen - 4  # a gradient of zero or of the other sign fails
