"""What the operator classes keep between calls: calls that need an earlier one, and the streams on
which a call's own memory is made and written."""
import pytest
import torch

import grouped_gemm_device_gb300 as g

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rows(M, N, dtype=BF, seed=0):
    gen = torch.Generator().manual_seed(seed)
    return torch.randn(M, N, generator=gen).to(dtype).cuda()


def test_layernorm_backward_needs_statistics(lib):
    ln, other = g.LayerNorm(64, 8), g.LayerNorm(64, 8)
    x, dy = rows(8, 64), rows(8, 64, seed=1)
    with pytest.raises(ValueError):
        ln.backward(dy, x)
    _, mean, rstd = other.forward(x)
    for kw in (dict(mean=mean), dict(rstd=rstd)):
        with pytest.raises(ValueError):
            ln.backward(dy, x, **kw)
    want = [t.clone() for t in other.backward(dy, x)]
    for a, b in zip(want, ln.backward(dy, x, mean=mean, rstd=rstd)):  # both given: no forward needed
        assert torch.equal(a, b)


def test_layernorm_backward_of_more_rows_than_the_forward_had(lib):
    ln = g.LayerNorm(64, 8)
    x, dy = rows(8, 64), rows(8, 64, seed=1)
    want = [t.clone() for t in (ln.forward(x)[0], *ln.backward(dy, x))]
    ln.forward(x[:4])
    with pytest.raises(ValueError):
        ln.backward(dy, x)
    with pytest.raises(ValueError):
        ln.backward(dy[:5], x[:5])
    for m in (4, 2):
        assert torch.equal(ln.backward(dy[:m], x[:m])[0], want[1][:m])


def test_router_loss_backward_needs_a_forward(lib):
    plan = g.RouterLoss(8, 2, 16)
    lg = rows(16, 8, torch.float32)
    ids = torch.topk(lg, 2).indices.int()
    with pytest.raises(ValueError):
        plan.backward(lg, ids)
    with pytest.raises(ValueError):
        plan.forward(lg, ids.long())
    with pytest.raises(ValueError):  # a refused forward is none
        plan.backward(lg, ids)
    plan.forward(lg, ids)
    whole = plan.backward(lg, ids).clone()
    assert whole.any()
    # a part of the tokens under the whole forward's counts
    assert torch.equal(plan.backward(lg[:5], ids[:5]), whole[:5])


def test_linear_backward_of_no_rows_writes_on_the_calls_stream(lib):
    lin = g.Fp8Linear(64, 64, 8)
    lin.set_weight(rows(64, 64))
    empty = torch.empty(0, 64, dtype=BF, device="cuda")
    for handle in (False, True):
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        stream = s.cuda_stream if handle else s
        lin.forward(empty, stream=stream)
        with torch.cuda.stream(s):
            torch.cuda._sleep(50_000_000)
            lin.dw.fill_(7.0)
        _, dw = lin.backward(empty, stream=stream)
        s.synchronize()
        torch.cuda.synchronize()
        assert not dw.any()


@pytest.mark.parametrize("handle", [False, True])
def test_layernorm_backward_makes_its_buffers_on_the_calls_stream(lib, handle):
    """Memory that the current stream has given back may still be in use there: a call on another
    stream does not take it."""
    M, N = 2048, 2048
    x, dy = rows(M, N), rows(M, N, seed=1)
    ln = g.LayerNorm(N, M)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = s.cuda_stream if handle else s
    ln.forward(x, stream=stream)
    freed = [torch.empty(M, N, dtype=BF, device="cuda") for _ in range(3)]
    held = [(t.data_ptr(), t.data_ptr() + 2 * M * N) for t in freed]
    del freed
    dx, dg, db = ln.backward(dy, x, stream=stream)
    s.synchronize()
    for lo, hi in held:
        assert not lo <= dx.data_ptr() < hi
    other = g.LayerNorm(N, M)
    other.forward(x)
    for a, b in zip((dx, dg, db), other.backward(dy, x)):
        assert torch.equal(a, b)


def test_clip_refuses_tensors_that_share_memory(lib):
    t = torch.ones(100, device="cuda")
    with pytest.raises(ValueError):
        g.GradClip([t, t]).clip(1.0)
    with pytest.raises(ValueError):
        g.GradClip([t[:60], t[40:]]).clip(1.0)
    with pytest.raises(ValueError):
        g.GradClip([t[:50]], [t[25:75]]).clip(1.0)
    assert torch.equal(t, torch.ones_like(t))
    # reading a tensor twice is a matter of the caller's norm
    assert abs(float(g.GradClip([t, t]).clip(float("inf"))) - 200 ** 0.5) <= 1e-5
    outs = [torch.empty_like(t), torch.empty_like(t)]
    g.GradClip([t, t], outs).clip(1.0)
    assert torch.equal(outs[0], outs[1])
    g.GradClip([t[:50], t[50:]]).clip(1.0)
    assert abs(float(t.norm()) - 1.0) <= 1e-5
