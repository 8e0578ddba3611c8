"""Objects made while their stream is busy, first called on another stream: what the constructors fill is
filled before the call."""
import math

import pytest
import torch

import grouped_gemm_device_gb300 as g

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def busy(make):
    """What `make` returns, made on a stream with some 50 ms of work before it, in memory that holds
    neither zeros nor what the object's tensors held before."""
    dirty = [torch.full((1 << s,), 0xA5, dtype=torch.uint8, device="cuda")
             for s in (9, 12, 16, 20, 22) for _ in range(8)]
    torch.cuda.synchronize()
    del dirty
    torch.cuda._sleep(100_000_000)
    return make()


def on_another_stream(call):
    """The call's tensors after it and everything else has ended."""
    s = torch.cuda.Stream()
    out = call(s)
    s.synchronize()
    torch.cuda.synchronize()
    return [t.clone() for t in out]


def same(make, call):
    torch.cuda.synchronize()
    want = [t.clone() for t in call(make(), None)]
    obj = busy(make)
    got = on_another_stream(lambda s: call(obj, s))
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("bits", [32, 8])
def test_adamw(lib, bits, handle):
    gen = torch.Generator().manual_seed(0)
    weights = [torch.randn(n, generator=gen).to(t).cuda() for n, t in ((5000, BF), (300, torch.float32))]
    grads = [torch.randn(w.shape, generator=gen).to(w.dtype).cuda() for w in weights]
    now = []

    def make():
        return g.AdamW(now, grads, state_bits=bits, seed=4)

    def call(opt, s):
        opt.step(stream=s.cuda_stream if handle and s else s)
        return [*opt.params, *opt.m, *opt.v, opt._counters, opt.masters[0]]

    now = [w.clone() for w in weights]
    want = [t.clone() for t in call(make(), None)]
    now = [w.clone() for w in weights]
    opt = busy(make)
    got = on_another_stream(lambda s: call(opt, s))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and int(opt.steps) == 1


def test_router_topk(lib):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(500, 64, generator=gen).cuda()
    same(lambda: g.RouterTopK(64, 4, 500), lambda plan, s: plan.forward(x, stream=s))


def test_router_loss(lib):
    gen = torch.Generator().manual_seed(2)
    x = torch.randn(500, 64, generator=gen).cuda()
    ids = torch.randint(0, 64, (500, 4), generator=gen, dtype=torch.int32).cuda()

    def call(loss, s):
        return [*loss.forward(x, ids, stream=s), loss.backward(x, ids, stream=s)]

    same(lambda: g.RouterLoss(64, 4, 500), call)


def test_grad_clip(lib):
    grads = [torch.full((5000,), 2.0, device="cuda"), torch.ones(77, device="cuda").to(BF)]
    same(lambda: g.GradClip(grads), lambda clip, s: [clip.clip(math.inf, stream=s)])


def test_fp8_linear(lib):
    gen = torch.Generator().manual_seed(3)
    w, x = (torch.randn(256, 256, generator=gen).to(BF).cuda() for _ in range(2))

    def call(linear, s):
        linear.set_weight(w, stream=s)
        return [linear.forward(x, stream=s), linear.err]

    same(lambda: g.Fp8Linear(256, 256, 256), call)


def test_layer_under_a_given_routing(lib):
    gen = torch.Generator().manual_seed(4)
    T, E, k, H, F = 200, 8, 2, 256, 256

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, generator=gen) * scale).to(BF).cuda()

    x, w1, w2 = rand(T, H), g.pack_w1(rand(E, H, 2 * F, scale=0.05)), rand(E, F, H, scale=0.05)
    ids = torch.randint(-1, E, (T, k), generator=gen, dtype=torch.int32).cuda()
    probs = torch.rand(T, k, generator=gen).cuda()

    def call(layer, s):
        layer.permute(ids, probs, x, stream=s)
        y = layer.forward(w1, w2, T, stream=s)
        return [y, layer.counts, layer.offsets()]

    same(lambda: g.MoELayer(g.make_desc(E=E, k=k, H=H, F=F, T_max=T)), call)


def test_memory_that_its_stream_still_writes(lib):
    """Buffers made of memory that was given back while the stream still writes it."""
    gen = torch.Generator().manual_seed(5)
    M, N = 512, 1024
    x, w = torch.randn(M, N, generator=gen).to(BF).cuda(), torch.ones(N, dtype=BF, device="cuda")

    def norm(plan, s):
        return [plan.forward(x, weight=w, stream=s)[1], plan.rstd]

    def layer_norm(plan, s):
        return plan.forward(x, w, stream=s)

    for make, call in ((lambda: g.ResidualNorm(N, M), norm), (lambda: g.LayerNorm(N, M), layer_norm)):
        want = [t.clone() for t in call(make(), None)]
        torch.cuda.synchronize()
        torch.cuda._sleep(100_000_000)
        late = [torch.full((M, N), 7.0, dtype=BF, device="cuda")]
        late += [torch.full((M,), 7.0, device="cuda") for _ in range(2)]
        del late
        plan = make()
        got = on_another_stream(lambda s: call(plan, s))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
