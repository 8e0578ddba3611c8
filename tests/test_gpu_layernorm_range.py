"""Layer norm's backward on rows whose spread is far from 1, where the third power of rstd leaves
fp32's range although rstd, its gradient and the forward do not."""
import pytest
import torch

import grouped_gemm_device_gb300 as g
from tests.test_gpu_layernorm import BF, F32, check_bwd, make

pytestmark = pytest.mark.gpu


# rstd^3 is subnormal from a spread of 4e12 on, 0 from 1e15 on; infinite below one of 1.4e-13
@pytest.mark.parametrize("spread,eps", [(1e14, 1e-5), (1e15, 1e-5), (1e17, 1e-5), (1e-13, 0.0),
                                        (1e-14, 0.0), (1e-17, 0.0)])
@pytest.mark.parametrize("N", [96, 1000, 1001, 4096, 16384, 20000])
@pytest.mark.parametrize("xt", [BF, F32])
def test_backward_of_rows_of_any_spread(lib, N, xt, spread, eps):
    M = 9
    x, dy, gamma, beta = make(M, N, xt, xt, mean=0.0, scale=spread)
    ln = g.LayerNorm(N, M, dtype=xt, eps=eps)
    _, mean, rstd = ln.forward(x, gamma, beta)
    check_bwd(dy, x, gamma, mean, rstd, ln.backward(dy, x, gamma))


def test_rows_of_different_spread_in_one_call(lib):
    M, N = 64, 1024
    x, dy, gamma, beta = make(M, N, F32, F32, mean=0.0)
    x *= 10.0 ** torch.linspace(-17, 17, M, device="cuda")[:, None]
    ln = g.LayerNorm(N, M, dtype=F32, eps=0.0)
    _, mean, rstd = ln.forward(x, gamma, beta)
    check_bwd(dy, x, gamma, mean, rstd, ln.backward(dy, x, gamma))
