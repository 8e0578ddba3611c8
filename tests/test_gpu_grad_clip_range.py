"""Clipping of finite gradients whose norm is above fp32's largest number, and of tensors that share
memory."""
import math

import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import block_ops as ob

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F32: 2.0 ** -24}


@pytest.mark.parametrize("n", [4, 1000, 2_000_003])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("max_norm", [1.0, 1e-6, 1e30])
def test_norm_above_the_largest_fp32(lib, n, dt, in_place, max_norm):
    gen = torch.Generator().manual_seed(n)
    a = (torch.rand(n, generator=gen) * 0.2 + 0.8).mul(3.3e38)
    a[::2] *= -1
    small = torch.tensor([1e-3, -2.0, 0.0, 1e20])
    grads = [a.to(dt).cuda(), small.cuda()]
    assert all(torch.isfinite(t).all() for t in grads)
    want = [t.double().cpu().numpy() for t in grads]
    norm, c = ob.clip(want, max_norm)
    assert norm > 3.4028235e38 and 0 < c < 1
    plan = g.GradClip(grads, None if in_place else [torch.full_like(t, 7.0) for t in grads])
    assert math.isinf(float(plan.clip(max_norm)))  # the norm's own rounding to fp32
    for w, o in zip(want, plan.outs):
        err = np.abs(o.double().cpu().numpy() - w * c)
        # the norm to 20 units of 2^-24, the factor's and the product's roundings, the result's own
        assert (err <= np.abs(w * c) * (HALF[o.dtype] * 1.01 + 24 * 2.0 ** -24) + 2.0 ** -134).all()


def test_infinite_elements_still_clip_the_rest_to_zero(lib):
    t = torch.full((100,), 3e38, device="cuda")
    t[7] = float("inf")
    out = torch.full_like(t, 7.0)
    assert math.isinf(float(g.GradClip([t], [out]).clip(1.0)))
    assert torch.isnan(out[7]) and not torch.cat([out[:7], out[8:]]).any()
