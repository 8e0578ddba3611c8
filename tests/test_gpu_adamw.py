"""AdamW with 32- and 8-bit states against the fp64 oracle; 8-bit codes bit by bit."""
import math

import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import step_ops as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24                       # half a step of fp32
B1, B2, EPS, LR = 0.9, 0.999, 1e-8, 1e-3
MIXES = [(F32, F32), (BF, BF), (BF, F32)]


def f64(t):
    return t.detach().double().cpu().numpy().reshape(-1)


def make(sizes, mixes, seed=0, scale=1e-2):
    gen = torch.Generator().manual_seed(seed)
    params = [(torch.randn(n, generator=gen) * 0.1).to(p).cuda() for n, (p, _) in zip(sizes, mixes)]
    grads = [(torch.randn(n, generator=gen) * scale).to(t).cuda() for n, (_, t) in zip(sizes, mixes)]
    return params, grads, gen


def new_grads(opt, gen, scale=1e-2):
    for t in opt.grads:
        t.copy_((torch.randn(t.shape, generator=gen) * scale).to(t.dtype))


class Twin:
    """The oracle's state beside an optimiser's: 32-bit states in fp64, 8-bit ones as codes."""

    def __init__(self, opt, decays):
        self.opt, self.decays, self.t = opt, decays, 0
        self.p = [f64(p if w is None else w) for p, w in zip(opt.params, opt.masters)]
        if opt.state_bits == 32:
            self.m = [np.zeros(p.shape) for p in self.p]
            self.v = [np.zeros(p.shape) for p in self.p]
        else:
            self.m = [so.encode(np.zeros(len(p), np.float32), np.zeros(len(p)), True)
                      for p in self.p]
            self.v = [so.encode(np.zeros(len(p), np.float32), np.zeros(len(p)), False)
                      for p in self.p]

    def step(self, norm=None, max_norm=math.inf):
        self.t += 1
        c = so.clip_factor(norm, max_norm)
        for i, (g_, decay) in enumerate(zip(self.opt.grads, self.decays)):
            gr = f64(g_)
            if self.opt.state_bits == 32:
                m, v = self.m[i], self.v[i]
            else:
                m, r = so.decode(*self.m[i], True), so.decode(*self.v[i], False)
                v = r * r
            self.p[i], m1, v1 = so.adamw(self.p[i], gr, m, v, self.t, LR, B1, B2, EPS, decay, c)
            if self.opt.state_bits == 32:
                self.m[i], self.v[i] = m1, v1
                continue
            g32 = gr.astype(np.float32) * c
            v32 = r.astype(np.float32) * r.astype(np.float32)
            m1, _, r1 = so.moments(g32, m, v32, B1, B2)
            w = so.words(self.opt.seed, self.t, i, len(gr))
            self.m[i] = so.encode(m1, (w & np.uint64(0xFFFF)).astype(np.int64), True)
            self.v[i] = so.encode(r1, (w >> np.uint64(16)).astype(np.int64), False)

    def check(self):
        """After n steps. m and v: a few roundings a step of terms that decay. A weight moves by about
        lr a step (at most 1 / (1 - beta1) of it), each move off by 20 U and by the rounding of the
        sum; the moments' errors move it by a like part."""
        n = self.t
        assert int(self.opt.steps) == n
        for i, p in enumerate(self.opt.params):
            got = f64(p if self.opt.masters[i] is None else self.opt.masters[i])
            tol = n * (U * np.abs(self.p[i]).max(initial=0) * 2 + 10 * LR * 40 * U)
            assert (np.abs(got - self.p[i]) <= tol).all()
            if self.opt.masters[i] is not None:
                assert torch.equal(p.reshape(-1), self.opt.masters[i].to(BF).reshape(-1))
            if self.opt.state_bits == 32:
                for mine, own in ((self.m[i], self.opt.m[i]), (self.v[i], self.opt.v[i])):
                    assert (np.abs(f64(own) - mine) <= 8 * n * U * np.abs(mine).max(initial=0)).all()
            else:
                for (c, s), codes, scales in ((self.m[i], self.opt.m[i], self.opt.m_exp[i]),
                                              (self.v[i], self.opt.v[i], self.opt.v_exp[i])):
                    assert (codes.cpu().numpy() == c).all() and (scales.cpu().numpy() == s).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[1], [256], [255, 257, 1, 0, 33], [4096, 100_003, 7]])
def test_steps(lib, bits, sizes):
    mixes = [MIXES[i % 3] for i in range(len(sizes))]
    decays = [0.1 * (i % 2) for i in range(len(sizes))]
    params, grads, gen = make(sizes, mixes)
    opt = g.AdamW(params, grads, lr=LR, betas=(B1, B2), eps=EPS, weight_decay=decays,
                  state_bits=bits, seed=(1 << 40) + 17)
    twin = Twin(opt, decays)
    for _ in range(4):
        opt.step()
        twin.step()
        twin.check()
        new_grads(opt, gen)


@pytest.mark.parametrize("bits", [32, 8])
def test_views_off_16_byte_boundaries(lib, bits):
    sizes = [3, 17, 1000, 8191, 1, 2, 30_007]
    total = sum(sizes)
    for pt, gt in MIXES:
        flat_p, flat_g, gen = make([total + 2], [(pt, gt)])
        flat_p, flat_g = flat_p[0], flat_g[0]
        keep = flat_p.clone()
        params, grads, at = [], [], 1
        for n in sizes:
            params.append(flat_p[at:at + n])
            grads.append(flat_g[at:at + n])
            at += n
        opt = g.AdamW(params, grads, lr=LR, weight_decay=0.1, state_bits=bits, seed=3)
        twin = Twin(opt, [0.1] * len(sizes))
        for _ in range(2):
            opt.step()
            twin.step()
        twin.check()
        assert torch.equal(flat_p[:1], keep[:1]) and torch.equal(flat_p[at:], keep[at:])


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(lib, bits):
    sizes = [(i * 37) % 501 for i in range(130)]
    params, grads, gen = make(sizes, [MIXES[i % 3] for i in range(130)])
    opt = g.AdamW(params, grads, lr=LR, state_bits=bits)
    twin = Twin(opt, [0.01] * 130)
    for _ in range(2):
        opt.step()
        twin.step()
    twin.check()


@pytest.mark.parametrize("bits", [32, 8])
def test_clipping_by_the_norm(lib, bits):
    sizes = [5000, 777]
    params, grads, gen = make(sizes, [(BF, BF), (F32, F32)], scale=1.0)
    opt = g.AdamW(params, grads, lr=LR, weight_decay=0.0, state_bits=bits)
    twin = Twin(opt, [0.0, 0.0])
    clip = g.GradClip(grads)
    for most in (1.0, 1e6):
        norm = clip.clip(math.inf)
        opt.step(norm=norm, max_norm=most)
        twin.step(float(norm), most)
        twin.check()
    # max_norm inf: the norm's finiteness alone counts
    opt.step(norm=norm)
    twin.step()
    twin.check()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_norm_that_is_not_finite_skips_the_step(lib, bits, bad):
    params, grads, _ = make([300, 4000], [(BF, BF), (F32, F32)])
    opt = g.AdamW(params, grads, lr=LR, state_bits=bits)
    clip = g.GradClip(grads)
    opt.step(norm=clip.clip(math.inf), max_norm=1.0)
    state = [*opt.params, *opt.m, *opt.v, *opt.m_exp, *opt.v_exp, *opt.masters, opt._counters]
    keep = [None if t is None else t.clone() for t in state]
    grads[0][5] = bad
    opt.step(norm=clip.clip(math.inf), max_norm=1.0)
    torch.cuda.synchronize()
    assert all(a is None or torch.equal(a, b) for a, b in zip(state, keep))
    grads[0][5] = 0.0
    opt.step(norm=clip.clip(math.inf), max_norm=1.0)
    assert int(opt.steps) == 2 and int(opt._counters[1]) == 0


def test_gradients_that_are_not_finite_without_a_norm(lib):
    """32 bits: the element alone; 8 bits: its block of 256."""
    for bits, hit in ((32, slice(300, 301)), (8, slice(256, 512))):
        params, grads, _ = make([1000], [(F32, F32)])
        grads[0][300] = math.inf
        opt = g.AdamW(params, grads, lr=LR, state_bits=bits)
        opt.step()
        assert not params[0][300].isfinite()
        rest = torch.ones(1000, dtype=torch.bool)
        rest[300] = False
        assert params[0].cpu()[rest].isfinite().all()
        m, v = (opt.m, opt.v) if bits == 32 else opt.moments()
        for t in (m[0], v[0]):
            bad = ~t.isfinite().cpu()
            assert bad[hit].all() and int(bad.sum()) == hit.stop - hit.start


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-8, 0.0])
@pytest.mark.parametrize("scale", [1e-16, 1e-19, 1e-30, 1e-4, 1e8, 1e15])
def test_far_magnitudes(lib, bits, eps, scale):
    """Gradients whose squares are subnormal, 0 or near fp32's end, and elements far below their
    block's largest: the codes are the oracle's, the weights move by lr where eps is 0."""
    gen = torch.Generator().manual_seed(2)
    params = [torch.zeros(5000, device="cuda")]
    grads = [torch.randn(5000, generator=gen).mul_(scale).cuda()]
    grads[0][::3] *= 1e-4
    grads[0][1000:1600] = 0
    grads[0][2048:2300] *= 2.0 ** -20
    opt = g.AdamW(params, grads, lr=LR, betas=(B1, B2), eps=eps, weight_decay=0.0, state_bits=bits)
    m = v = np.zeros(5000)
    codes = None
    for t in range(1, 4):
        gr = f64(grads[0])
        r = None
        if bits == 8 and codes is not None:
            m, r = so.decode(*codes[0], True), so.decode(*codes[1], False)
        m32 = m.astype(np.float32)
        v32 = v.astype(np.float32) if r is None else r.astype(np.float32) * r.astype(np.float32)
        with np.errstate(under="ignore"):
            m1, v1, r1 = so.moments(gr.astype(np.float32), m32, v32, B1, B2)
        before = f64(params[0])
        opt.step()
        if bits == 8:
            w = so.words(0, t, 0, 5000)
            codes = (so.encode(m1, (w & np.uint64(0xFFFF)).astype(np.int64), True),
                     so.encode(r1, (w >> np.uint64(16)).astype(np.int64), False))
            for (c, s), own, scales in zip(codes, (opt.m, opt.v), (opt.m_exp, opt.v_exp)):
                assert (own[0].cpu().numpy() == c).all() and (scales[0].cpu().numpy() == s).all()
        else:
            # the same roundings, whatever the path
            assert (f64(opt.m[0]) == m1).all() and (f64(opt.v[0]) == v1).all()
            m, v = m1.astype(np.float64), v1.astype(np.float64)
        # r32 is the rounded root; the move is off by a few roundings of itself and of the weight
        with np.errstate(invalid="ignore", divide="ignore"):  # 0 / 0 where nothing has been seen
            c1, c2 = 1 - B1 ** t, 1 - B2 ** t
            move = LR / c1 * m1.astype(np.float64) / (r1.astype(np.float64) / c2 ** 0.5 + eps)
        after = f64(params[0])
        ok = np.isfinite(move)
        assert (~ok == ((r1 == 0) & (eps == 0))).all()
        assert (np.abs(after[ok] - (before[ok] - move[ok])) <= 40 * U * np.abs(move[ok])
                + 2 * U * np.abs(before[ok])).all()
        params[0].zero_()   # 0 / 0 where nothing has been seen and eps is 0


def test_moments(lib):
    """Every code under several scales, the smallest and the largest among them."""
    params, grads, _ = make([2000, 5], [(F32, F32)] * 2)
    opt = g.AdamW(params, grads, state_bits=8)
    gen = torch.Generator().manual_seed(1)
    for name, signed in (("m", True), ("v", False)):
        codes, scales = getattr(opt, name)[0], getattr(opt, name + "_exp")[0]
        codes.copy_(torch.randint(0, 256, codes.shape, generator=gen, dtype=torch.uint8))
        scales.copy_(torch.tensor([32, 33, 100, 127, 200, 254, 255, 40], dtype=torch.uint8))
    m, v = opt.moments()
    for name, t, signed in (("m", m[0], True), ("v", v[0], False)):
        want = so.decode(getattr(opt, name)[0].cpu().numpy(),
                         getattr(opt, name + "_exp")[0].cpu().numpy(), signed)
        assert np.array_equal(f64(t), want, equal_nan=True)
    assert not m[1].any() and not v[1].any()


def test_states_follow_a_long_run(lib):
    """2000 steps of gradients of unit variance: 8-bit states stay near the 32-bit ones. r = sqrt(v)
    decays by 1 / 2000 a step, which rounding to the nearest code would lose. A step of r / 11 is
    taken with probability 11 / 2000: variance r^2 / (11 * 2000) a step, over a memory of 1000 steps
    (r follows v, whose memory is 1000): relative spread of about sqrt(1000 / 22000 / 2) = 0.15 an
    element; the mean over 4096 elements is off by a 64th of it and by the square's bias (half of
    0.15^2)."""
    outs = []
    for bits in (32, 8):
        params, grads, gen = make([4096], [(F32, F32)])
        opt = g.AdamW(params, grads, lr=0.0, state_bits=bits, seed=5)
        gpu = torch.Generator(device="cuda").manual_seed(7)
        for _ in range(2000):
            grads[0].normal_(generator=gpu)
            opt.step()
        outs.append(opt.v[0].sqrt() if bits == 32 else opt.moments()[1][0].float())
    ratio = (outs[1] / outs[0]).cpu()
    assert abs(float(ratio.mean()) - 1) < 0.05 and float(ratio.std()) < 0.3


def test_learning_rate_and_steps_in_a_captured_step(lib):
    params, grads, _ = make([10_000, 300], [(BF, BF), (F32, F32)])
    twins = []
    for graph_used in (False, True):
        ps, gs = [p.clone() for p in params], [t.clone() for t in grads]
        lr = torch.full((1,), LR, device="cuda")
        opt = g.AdamW(ps, gs, lr=lr, state_bits=8, seed=9)
        clip = g.GradClip(gs)

        def step():
            opt.step(norm=clip.clip(math.inf), max_norm=0.5)

        step()
        if graph_used:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            again = graph.replay
        else:
            again = step
        for k in range(4):
            lr.fill_(LR / (k + 1))
            again()
        torch.cuda.synchronize()
        assert int(opt.steps) == 5
        twins.append([*ps, *opt.m, *opt.v, *opt.m_exp, *opt.v_exp])
    assert all(torch.equal(a, b) for a, b in zip(*twins))


def test_resumed_run_goes_on_alike(lib):
    params, grads, gen = make([5000, 70], [(BF, BF), (F32, F32)])
    opt = g.AdamW(params, grads, lr=LR, state_bits=8, seed=1)
    for _ in range(3):
        opt.step()
    ps, gs = [p.clone() for p in params], [t.clone() for t in grads]
    two = g.AdamW(ps, gs, lr=LR, state_bits=8, seed=1)
    for name in ("m", "v", "m_exp", "v_exp", "masters"):
        for a, b in zip(getattr(two, name), getattr(opt, name)):
            if a is not None:
                a.copy_(b)
    two.steps.copy_(opt.steps)
    opt.step()
    two.step(stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    for a, b in zip([*ps, *two.m, *two.v], [*params, *opt.m, *opt.v]):
        assert torch.equal(a, b)


def test_no_tensors_still_counts_the_step(lib):
    opt = g.AdamW([], [])
    opt.step()
    opt.step()
    assert int(opt.steps) == 2


def test_argument_checks(lib):
    p, gr = torch.zeros(8, 4, device="cuda"), torch.zeros(8, 4, device="cuda")
    for f in (lambda: g.AdamW([p], []), lambda: g.AdamW([p], [gr.t()]),
              lambda: g.AdamW([p.cpu()], [gr]), lambda: g.AdamW([p], [gr[:4]]),
              lambda: g.AdamW([p.half()], [gr]), lambda: g.AdamW([p], [gr.half()]),
              lambda: g.AdamW([p], [gr], state_bits=4), lambda: g.AdamW([p], [gr], seed=-1), lambda: g.AdamW([p], [gr], masters=[gr]),
              lambda: g.AdamW([p.to(BF)], [gr], masters=[p.to(BF)]),
              lambda: g.AdamW([p], [gr], weight_decay=[0.1, 0.2]), lambda: g.AdamW([p], [p]),
              lambda: g.AdamW([p, p], [gr, gr]), lambda: g.AdamW([p, p[:4]], [gr, gr[:4]])):
        with pytest.raises(ValueError):
            f()
    opt = g.AdamW([p], [gr])
    for f in (lambda: opt.step(max_norm=1.0), lambda: opt.step(norm=torch.zeros(2, device="cuda")),
              lambda: opt.step(norm=torch.zeros(1)), lambda: opt.moments(),
              lambda: opt.step(lr=torch.zeros(1, device="cuda", dtype=BF))):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(g.MoeError):
        opt.step(lr=-1.0)
    # one gradient for two weights is the caller's matter
    g.AdamW([p, torch.zeros(8, 4, device="cuda")], [gr, gr]).step()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-6, 1e-12, 1e-30, 1e-42, 1e36, 1e38, 2.9e38])
@pytest.mark.parametrize("scale", [0.0, 1e-22, 1e-19, 1e-4, 1e15])
def test_far_denominators(lib, bits, eps, scale):
    """Denominators from subnormal numbers to fp32's end: elements that have seen no gradient stay, the
    others move as the formula says, whatever path their places take."""
    n = 5000
    gen = torch.Generator().manual_seed(6)
    params = [torch.zeros(n, device="cuda"), torch.zeros(n + 1, device="cuda")[1:]]
    grads = [torch.randn(n, generator=gen).mul_(scale).cuda() for _ in params]
    for t in grads:
        t[::3] *= 1e-4
        t[1000:1600] = 0
    opt = g.AdamW(params, grads, lr=LR, betas=(B1, B2), eps=eps, weight_decay=0.0, state_bits=bits)
    opt.step()
    held = float(np.float32(eps))
    zero = np.zeros(n, np.float32)
    for p, t in zip(params, grads):
        with np.errstate(under="ignore"):
            m, _, r = so.moments(f64(t).astype(np.float32), zero, zero, B1, B2)
        m, r = m.astype(np.float64), r.astype(np.float64)
        move = LR / (1 - B1) * m / (r / (1 - B2) ** 0.5 + held)
        # lr, its correction (a product, expm1's two steps, a quotient), the root's correction (as many
        # and a root), the approximate root and reciprocal (2 U each), two products, a sum: 20 U; what
        # is below 2^-126 has steps of 2^-149, in the quotient and in its product with lr
        assert (np.abs(f64(p) + move) <= 20 * U * np.abs(move) + 2.0 ** -148).all()
        assert not f64(p)[1000:1600].any()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-44, 1e-45, 1e-50, 5e-324])
def test_an_eps_below_fp32_is_not_0(lib, bits, eps):
    """What has seen no gradient stays where it is; what has seen one moves by lr."""
    params = [torch.full((3000,), 0.5, device="cuda") for _ in range(2)]
    grads = [torch.zeros(3000, device="cuda") for _ in range(2)]
    grads[1][::2] = 1e-3
    opt = g.AdamW(params, grads, lr=LR, betas=(B1, B2), eps=eps, weight_decay=0.0, state_bits=bits)
    for t in (1, 2):
        opt.step()
        assert (params[0] == 0.5).all() and (params[1][1::2] == 0.5).all()
    # two moves of lr, each off by 20 U and the rounding of the sum, m and r held exactly or (8 bits) to
    # an eighth after the first step
    off = np.abs(f64(params[1][::2]) - (0.5 - 2 * LR))
    assert (off <= 2 * (20 * U * LR + U * 0.5) + (0.25 * LR if bits == 8 else 0.0)).all()
