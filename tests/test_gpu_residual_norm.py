"""The residual stream around a block and its norms against the fp64 oracle."""
import numpy as np
import pytest
import torch

import grouped_gemm_device_gb300 as g
from oracle import step_ops as so

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24                       # half a step of fp32
HALF = {BF: 2.0 ** -8, F32: U}       # half a step, relative
TYPES = [(BF, BF, BF), (BF, BF, F32), (F32, BF, F32), (F32, BF, BF), (F32, F32, F32)]
EPS, SCALE = 1e-5, 0.7


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rows_of(M, N, dtype, gen, scale=1.0, lay="plain"):
    t = (torch.randn(M, N, generator=gen) * scale).to(dtype)
    if lay == "plain":
        return t.cuda()
    pad = {"wide": (0, 16), "odd": (3, 4), "shift": (1, 8)}[lay]
    buf = torch.full((M, N + sum(pad)), 9.0, dtype=dtype, device="cuda")
    buf[:, pad[0]:pad[0] + N] = t.cuda()
    return buf[:, pad[0]:pad[0] + N]


class Case:
    """One block's inputs, results of both passes and what they should be."""

    def __init__(self, M, N, types, branch=True, post=True, gate=True, weights=True, norm=True,
                 grad_h=True, grad_x=True, lay="plain", seed=0):
        xt, ot, wt = types
        gen = torch.Generator().manual_seed(seed)
        self.x = rows_of(M, N, xt, gen, 1.5, lay)
        self.o = rows_of(M, N, ot, gen, 0.7, lay) if branch else None
        self.w = (1 + 0.2 * torch.randn(N, generator=gen)).to(wt).cuda() if weights and norm else None
        self.wp = ((1 + 0.2 * torch.randn(N, generator=gen)).to(wt).cuda() if weights and branch
                   else None)
        self.gate = torch.rand(M, generator=gen).cuda() if gate and branch else None
        self.dh = rows_of(M, N, ot, gen, 1.0, lay) if norm and grad_h else None
        self.dx_new = rows_of(M, N, xt, gen, 1.0, lay) if grad_x or self.dh is None else None
        self.post, self.norm, self.N = post and branch, norm, N
        self.plan = g.ResidualNorm(N, M + 2, dtype=xt, branch_dtype=ot, weight_dtype=wt,
                                   post_norm=post, scale=SCALE, eps=EPS)

    def forward(self, **kw):
        return self.plan.forward(self.x, self.o, self.w, self.wp, self.gate, self.norm, **kw)

    def backward(self, x_new, **kw):
        w = self.w if self.dh is not None else None
        return self.plan.backward(self.dh, x_new, self.o, w, self.wp, self.gate, self.dx_new, **kw)

    # A sum over a row: a thread's own additions (N / 32 at most), then a tree; the mean, eps, root and
    # reciprocal: 1 or 2 each
    def row_tol(self):
        return (self.N / 32 + 20) * U

    def check(self):
        x_new, h = self.forward()
        d = self.backward(x_new)
        torch.cuda.synchronize()
        x, o, gate, wp, w = (f64(t) for t in (self.x, self.o, self.gate, self.wp, self.w))
        new = f64(x_new)
        if self.o is None:
            assert x_new is self.x
        else:
            want = so.residual(x, o, wp, gate, SCALE, self.post, EPS)
            part = np.abs(want - x)
            tol = HALF[x_new.dtype] * np.abs(want) * 1.01 + (self.row_tol() + 8 * U) * part
            assert (np.abs(new - want) <= tol + U * np.abs(x) + 2.0 ** -133).all()
        if self.norm:
            want = so.normed(new, w, EPS)  # of the stream as it is stored
            tol = (HALF[h.dtype] * 1.01 + self.row_tol() + 8 * U) * np.abs(want)
            assert (np.abs(f64(h) - want) <= tol + 2.0 ** -133).all()
        else:
            assert h is None
        ref = so.residual_grad(f64(self.dh), f64(self.dx_new), new, o, wp, gate,
                               w if self.dh is not None else None, SCALE, self.post, EPS)
        M = len(x)
        for name, got in zip(("dx", "do", "d_weight", "d_post_weight", "d_gate"), d):
            if got is None:
                assert {"do": self.o, "d_weight": self.w if self.dh is not None else None,
                        "d_post_weight": self.wp, "d_gate": self.gate}[name] is None
                continue
            want, size = ref[name]
            # three sums over rows lie behind a value; a weight's gradient adds a block's rows one
            # by one (at most all of them), then 480 partials in 15 + 5 steps
            more = (M + 20) * U if name.endswith("weight") else 0.0
            tol = (3 * self.row_tol() + 16 * U + more) * size + HALF[got.dtype] * np.abs(want) * 1.01
            assert (np.abs(f64(got) - want) <= tol + 2.0 ** -133).all(), name
        return x_new, h, d


SIZES = [(1, 1), (3, 7), (1, 4096), (5, 64), (33, 33), (100, 127), (17, 256), (64, 1000), (9, 2880),
         (300, 513), (7, 4095), (40, 5120), (3, 7168), (4, 16384), (2, 40001)]


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("size", SIZES)
def test_both_passes(lib, size, types):
    Case(*size, types).check()
    Case(*size, types, post=False, gate=False).check()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("kw", [
    dict(branch=False), dict(branch=False, grad_x=False), dict(branch=False, weights=False),
    dict(norm=False), dict(norm=False, post=False), dict(weights=False), dict(grad_x=False),
    dict(gate=False), dict(post=False), dict(post=False, weights=False, gate=False),
    dict(grad_h=False)])
def test_parts_left_out(lib, types, kw):
    Case(50, 384, types, **kw).check()
    Case(20, 131, types, **kw).check()


@pytest.mark.parametrize("lay", ["wide", "odd", "shift"])
@pytest.mark.parametrize("types", TYPES)
def test_strides_and_places(lib, lay, types):
    for N in (1000, 129, 4096):
        Case(21, N, types, lay=lay).check()


@pytest.mark.parametrize("types", TYPES)
@pytest.mark.parametrize("N", [64, 1024, 2047, 4096])
def test_many_rows(lib, types, N):
    Case(2500, N, types).check()


@pytest.mark.parametrize("types", [(BF, BF, BF), (F32, BF, F32), (F32, F32, F32)])
@pytest.mark.parametrize("N", [249, 255, 505, 511, 1019, 1023, 2041, 2047, 4089, 4093, 4095, 8191])
def test_rows_that_wrap(lib, types, N):
    """Rows just below a group's columns, many (whose groups walk rows) and few, at every place."""
    Case(700, N, types).check()
    Case(11, N, types, post=False, gate=False).check()


def test_rows_of_zeros_and_far_magnitudes(lib):
    c = Case(6, 512, (F32, F32, F32))
    c.x[0] = 0
    c.o[:2] = 0
    c.x[2] *= 1e12
    c.o[3] *= 1e-12
    c.x[4] *= 1e-12
    c.check()


def test_infinities_and_nan_stay_in_their_row(lib):
    c = Case(6, 256, (BF, BF, BF))
    want = [t.clone() for t in c.forward()]
    c.x[1, 7] = float("nan")
    c.o[2, 200] = float("inf")
    x_new, h = c.forward()
    for a, b in zip((x_new, h), want):
        keep = [0, 3, 4, 5]
        assert torch.equal(a[keep], b[keep])
        assert a[1].isnan().any() and not a[2].isfinite().all()


def test_in_place(lib):
    M, N = 37, 520
    gen = torch.Generator().manual_seed(4)
    x, o, dh, dxn = (rows_of(M, N, BF, gen) for _ in range(4))
    w, wp = (1 + 0.1 * torch.randn(2, N, generator=gen)).to(BF).cuda()
    gate = torch.rand(M, generator=gen).cuda()
    plan = g.ResidualNorm(N, M, post_norm=True)
    x_new, h = plan.forward(x, o, w, wp, gate)
    dx, do = plan.backward(dh, x_new, o, w, wp, gate, dxn)[:2]
    x2, o2, r = x.clone(), o.clone(), torch.empty(2, M, device="cuda")
    g.moe_residual_norm_fwd(x2, N, o2, N, wp, gate, w, x2, N, o2, N, r[0], r[1], M, N, 1.0, 1, 1e-6,
                            0, 0, 0)
    assert torch.equal(x2, x_new) and torch.equal(o2, h)
    for at in ("dh", "o"):
        a = dict(dh=dh.clone(), o=o.clone(), dx=dxn.clone())
        g.moe_residual_norm_bwd(a["dh"], N, a["dx"], N, x_new, N, a["o"], N, wp, gate, w, r[0], r[1],
                                a["dx"], N, a[at], N, None, None, None, M, N, 1.0, 1, 0, 0, 0, None,
                                0)
        assert torch.equal(a["dx"], dx) and torch.equal(a[at], do)


def test_rows_behind_the_last_stay_and_no_rows(lib):
    plan = g.ResidualNorm(64, 10, post_norm=True)
    gen = torch.Generator().manual_seed(5)
    x, o = rows_of(10, 64, BF, gen), rows_of(10, 64, BF, gen)
    w = torch.ones(64, dtype=BF, device="cuda")
    x_new, h = plan.forward(x, o, w, w)
    plan.backward(h, x_new, o, w, w)
    keep = [t.clone() for t in (plan.x_new, plan.h, plan.dx, plan.do, plan.rstd)]
    x_new, h = plan.forward(o[:4], x[:4], w, w)
    plan.backward(h, x_new, x[:4], w, w)
    for a, b in zip((plan.x_new, plan.h, plan.dx, plan.do, plan.rstd), keep):
        assert torch.equal(a[4:], b[4:]) and not torch.equal(a[:4], b[:4])
    x_new, h = plan.forward(x[:0], o[:0], w, w)
    dx, do, dw, dwp, dg = plan.backward(h, x_new, o[:0], w, w)
    assert x_new.shape == dx.shape == (0, 64) and dg is None
    assert not dw.any() and not dwp.any()


def test_same_results_again_in_a_graph_and_on_another_stream(lib):
    c = Case(700, 2048, (BF, BF, BF))

    def call(**kw):
        x_new, h = c.forward(**kw)
        return x_new, h, *c.backward(x_new, **kw)

    want = [t.clone() for t in call()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs = call()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, outs))
    for stream in (s, s.cuda_stream):
        outs = call(stream=stream)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, outs))


@pytest.mark.parametrize("handle", [False, True])
def test_buffers_are_made_on_the_calls_stream(lib, handle):
    M, N = 1024, 2048
    c = Case(M, N, (BF, BF, BF))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    stream = s.cuda_stream if handle else s
    freed = [torch.empty(M + 2, N, dtype=BF, device="cuda") for _ in range(4)]
    held = [(t.data_ptr(), t.data_ptr() + 2 * (M + 2) * N) for t in freed]
    del freed
    x_new, _ = c.forward(stream=stream)
    outs = x_new, *c.backward(x_new, stream=stream)[:2]
    s.synchronize()
    for t in outs:
        assert not any(lo <= t.data_ptr() < hi for lo, hi in held)


def test_argument_checks(lib):
    plan = g.ResidualNorm(64, 8, post_norm=True)
    x, w = torch.zeros(8, 64, dtype=BF, device="cuda"), torch.ones(64, dtype=BF, device="cuda")
    gate = torch.ones(8, device="cuda")
    with pytest.raises(ValueError):
        plan.backward(x, x, x, w, w)     # no forward yet
    plan.forward(x[:4], x[:4], w, w)
    for f in (lambda: plan.backward(x, x, x, w, w), lambda: plan.forward(x.float(), x, w, w),
              lambda: plan.forward(x, x[:4], w, w), lambda: plan.forward(x, x, w.float(), w),
              lambda: plan.forward(x, None, w, w), lambda: plan.forward(x, None, w, None, gate),
              lambda: plan.forward(x, x, w, w, gate.to(BF)), lambda: plan.forward(x, x, w, w, gate[:4]),
              lambda: plan.forward(x, x, w, norm=False), lambda: plan.forward(x, norm=False),
              lambda: plan.forward(x.cpu(), x, w, w), lambda: plan.forward(x[:, :32], x, w, w),
              lambda: plan.forward(torch.zeros(9, 64, dtype=BF, device="cuda")),
              lambda: plan.backward(None, None, x), lambda: plan.backward(x[:4], None, x[:4], w),
              lambda: plan.backward(None, x, x[:4], w, dx_new=x[:4]),
              lambda: plan.backward(x[:4], x, x[:4], w, w),
              lambda: plan.backward(x[:4], x[:4], x, w, w),
              lambda: plan.backward(x[:4], x[:4], x[:4], w, w, dx_new=x),
              lambda: plan.backward(x[:4], x[:4], x[:4], w, w, rstd=gate),
              lambda: g.ResidualNorm(64, 8, dtype=torch.float16)):
        with pytest.raises(ValueError):
            f()
    with pytest.raises(g.MoeError):
        g.ResidualNorm(64, 8, dtype=BF, branch_dtype=F32).forward(x, x.float())


@pytest.mark.parametrize("types", [(BF, BF, BF), (F32, BF, F32), (F32, F32, F32)])
@pytest.mark.parametrize("N", [7, 512, 513, 520, 1019, 2880, 4095, 4096, 8192, 9000])
def test_a_workspace_on_any_16_byte_boundary(lib, types, N):
    """The weights' gradients through partial sums in a workspace at every 16 bytes of a 64: the same
    bits, and nothing written outside the bytes that the call asks for."""
    xt, ot, wt = types
    for M in (2, 40):
        c = Case(M, N, types)
        x_new, _ = c.forward()
        want = [t.clone() for t in c.backward(x_new)]
        need = g.moe_residual_norm_workspace(M, N)
        code = {BF: 0, F32: 1}
        outs = [torch.empty_like(t) for t in want]
        dx, do, dw, dwp, dg = outs
        for at in (0, 16, 32, 48):
            buf = torch.full((need + 128,), 0x5A, dtype=torch.uint8, device="cuda")
            assert buf.data_ptr() % 64 == 0
            for t in outs:
                t.fill_(7.0)
            g.moe_residual_norm_bwd(c.dh, N, c.dx_new, N, x_new, N, c.o, N, c.wp, c.gate, c.w,
                                    c.plan.rstd_post, c.plan.rstd, dx, N, do, N, dwp, dw, dg, M, N,
                                    SCALE, 1, code[xt], code[ot], code[wt], buf.data_ptr() + at, need)
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
            assert (buf[:at] == 0x5A).all() and (buf[at + need:] == 0x5A).all()


def test_rows_of_its_own_buffers(lib):
    """The stream goes on in the class's own buffers, row for row; other rows of them are refused."""
    gen = torch.Generator().manual_seed(9)
    M, N = 12, 264
    x, o, dh = (rows_of(M, N, BF, gen) for _ in range(3))
    w = (1 + 0.1 * torch.randn(N, generator=gen)).to(BF).cuda()
    plan, other = (g.ResidualNorm(N, M, post_norm=True) for _ in range(2))
    first = other.forward(x, o, w, w)[0].clone()
    want = [t.clone() for t in other.forward(first, o, w, w)]
    got = plan.forward(plan.forward(x, o, w, w)[0], o, w, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    grads = [t.clone() for t in other.backward(dh, want[0], o, w, w)[:2]]
    back = plan.backward(dh, want[0], o, w, w)[:2]
    assert all(torch.equal(a, b) for a, b in zip(back, grads))
    more = [t.clone() for t in other.backward(grads[1], want[0], o, w, w, dx_new=grads[0])[:2]]
    back = plan.backward(plan.do, want[0], o, w, w, dx_new=plan.dx)[:2]
    assert all(torch.equal(a, b) for a, b in zip(back, more))
    for f in (lambda: plan.forward(plan.x_new[1:], o[1:], w, w),
              lambda: plan.forward(x[3:], plan.x_new[3:], w, w),
              lambda: plan.forward(plan.h[1:4], weight=w),
              lambda: plan.backward(plan.do[1:], want[0][1:], o[1:], w, w),
              lambda: plan.backward(dh[1:], want[0][1:], o[1:], w, w, dx_new=plan.dx[1:])):
        with pytest.raises(g.MoeError):
            f()
    # rows behind those that are written are any
    got = plan.forward(plan.x_new[6:], o[6:], w, w)
    want = other.forward(want[0][6:], o[6:], w, w)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
