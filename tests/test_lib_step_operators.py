"""CPU-only checks of the step's operators: the refusals of their host-side checks, workspace sizes and
the layout of the AdamW list (none of these calls touches the device)."""
import ctypes
import math
import os
import subprocess

import pytest

import grouped_gemm_device_gb300 as g
from grouped_gemm_device_gb300 import build as gbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20  # a plausible, well-aligned address that is never followed
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def lib():
    gbuild.build()
    return g.load()


def refused(fn, status, base, **change):
    args = dict(base, **change)
    with pytest.raises(g.MoeError) as e:
        fn(**args)
    assert e.value.status == status, str(e.value)
    assert len(str(e.value)) > 12


TOPK = dict(logits=P, ld_logits=8, logits_dtype=1, bias=P, token_mask=None, T=4, E=8, k=2, score=1,
            n_group=4, topk_group=2, group_top=2, renorm=1, scale=1.0, topk_ids=P, topk_weights=P,
            counts=P, stream=0)


@pytest.mark.parametrize("change", [
    dict(E=0), dict(E=257, ld_logits=257, n_group=1, topk_group=1), dict(k=0), dict(k=9),
    dict(k=5), dict(T=-1), dict(ld_logits=7), dict(logits_dtype=2), dict(score=2), dict(score=-1),
    dict(n_group=0), dict(n_group=3), dict(topk_group=0), dict(topk_group=5), dict(group_top=0),
    dict(group_top=3), dict(n_group=8, topk_group=8), dict(logits=None), dict(topk_ids=None),
    dict(topk_weights=None), dict(logits=P + 2), dict(bias=P + 1), dict(counts=P + 2),
    dict(topk_ids=P + 2), dict(n_group=4, topk_group=1, k=3)])
def test_router_topk_forward_refuses(change):
    refused(g.moe_router_topk_fwd, INVALID, TOPK, **change)


def test_router_topk_backward_refuses():
    base = dict(logits=P, ld_logits=8, logits_dtype=0, topk_ids=P, d_weights=P, T=4, E=8, k=2,
                score=0, renorm=0, scale=1.0, add_to=None, ld_add=0, d_logits=P, ld_d=8, stream=0)
    for change in (dict(E=0), dict(k=9), dict(T=-1), dict(ld_logits=7), dict(ld_d=7),
                   dict(add_to=P, ld_add=7), dict(add_to=P, ld_add=16), dict(logits=None),
                   dict(topk_ids=None), dict(d_weights=None), dict(d_logits=None),
                   dict(logits=P + 1), dict(d_weights=P + 2), dict(add_to=P + 2, ld_add=8),
                   dict(logits_dtype=5), dict(score=7)):
        refused(g.moe_router_topk_bwd, INVALID, base, **change)


FWD = dict(x=P, ldx=64, o=P, ldo=64, post_weight=P, gate=P, weight=P, x_new=P, ldxn=64, h=P,
           ldh=64, rstd_post=P, rstd=P, M=4, N=64, scale=1.0, post_norm=1, eps=1e-6, x_dtype=0,
           o_dtype=0, w_dtype=0, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(ldx=63), INVALID), (dict(ldo=63), INVALID),
    (dict(ldxn=63), INVALID), (dict(ldh=63), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID), (dict(x=None, x_new=2 * P), INVALID), (dict(o=None), INVALID),
    (dict(x_new=None), INVALID), (dict(o=None, x_new=None), INVALID),
    (dict(o=None, x_new=None, post_weight=None, gate=None), INVALID),
    (dict(h=None), INVALID), (dict(ldxn=128), INVALID), (dict(h=P, ldh=128), INVALID),
    (dict(o=None, x_new=None, post_weight=None, gate=None, post_norm=0, h=None, weight=None),
     INVALID),
    (dict(x=P + 1), INVALID), (dict(h=P + 1), INVALID), (dict(gate=P + 2), INVALID),
    (dict(weight=P + 1), INVALID), (dict(rstd=P + 2), INVALID), (dict(x_dtype=2), INVALID),
    (dict(w_dtype=-1), INVALID), (dict(x_dtype=0, o_dtype=1), UNSUPPORTED),
    (dict(x_dtype=1, o_dtype=1, w_dtype=0), UNSUPPORTED),
    (dict(N=1 << 31, ldx=1 << 31, ldo=1 << 31, ldxn=1 << 31, ldh=1 << 31), UNSUPPORTED)])
def test_residual_norm_forward_refuses(change, status):
    refused(g.moe_residual_norm_fwd, status, FWD, **change)


BWD = dict(dh=P, lddh=64, dx_new=P, lddxn=64, x_new=P, ldxn=64, o=P, ldo=64, post_weight=P, gate=P,
           weight=P, rstd_post=P, rstd=P, dx=P, lddx=64, d_o=P, lddo=64, d_post_weight=P,
           d_weight=P, d_gate=P, M=4, N=64, scale=1.0, post_norm=1, x_dtype=0, o_dtype=0,
           w_dtype=0, ws=P, ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(dh=None, dx_new=None), INVALID),
    (dict(dh=None), INVALID), (dict(x_new=None), INVALID), (dict(rstd=None), INVALID),
    (dict(o=None), INVALID), (dict(rstd_post=None), INVALID), (dict(gate=None), INVALID),
    (dict(post_weight=None), INVALID), (dict(ws=None), INVALID), (dict(ws=P + 8), INVALID),
    (dict(ws_bytes=64), WORKSPACE), (dict(lddh=63), INVALID), (dict(lddxn=63), INVALID),
    (dict(ldxn=63), INVALID), (dict(ldo=63), INVALID), (dict(lddx=63), INVALID),
    (dict(lddo=63), INVALID), (dict(lddx=128), INVALID), (dict(lddo=128), INVALID),
    (dict(dh=P + 1), INVALID), (dict(d_gate=P + 2), INVALID), (dict(d_weight=P + 1), INVALID),
    (dict(x_dtype=3), INVALID), (dict(o_dtype=1), UNSUPPORTED),
    (dict(dx=None, d_o=None, d_weight=None, d_post_weight=None, d_gate=None), INVALID)])
def test_residual_norm_backward_refuses(change, status):
    refused(g.moe_residual_norm_bwd, status, BWD, **change)


def test_residual_norm_workspace():
    a, b, c = (g.moe_residual_norm_workspace(*s) for s in ((1, 64), (100, 64), (100, 128)))
    assert 0 < a <= b <= c and g.moe_residual_norm_workspace(0, 1) > 0
    for bad in ((1, 0), (-1, 4), (1 << 31, 4)):
        with pytest.raises(g.MoeError):
            g.moe_residual_norm_workspace(*bad)


def adamw_args(**kw):
    base = dict(param=P, master=2 * P, grad=3 * P, m=4 * P, v=5 * P, m_scale=6 * P, v_scale=7 * P,
                numel=4, param_dtype=0, grad_dtype=0, decay=0.1, reserved=0)
    base.update(kw)
    return dict(n=1, tensors=(g.AdamWTensor * 1)(g.AdamWTensor(**base)), state_bits=8, lr=1e-3,
                lr_device=None, beta1=0.9, beta2=0.999, eps=1e-8, grad_norm=None, max_norm=1.0,
                seed=0, counters=P, stream=0)


def test_adamw_refuses():
    base = adamw_args()
    for change in (dict(n=-1), dict(n=65537), dict(tensors=None), dict(state_bits=16),
                   dict(lr=-1.0), dict(lr=math.inf), dict(lr=math.nan), dict(eps=-1e-8),
                   dict(eps=math.nan), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.5),
                   dict(beta2=math.nan), dict(max_norm=0.0), dict(max_norm=math.nan),
                   dict(counters=None), dict(counters=P + 4), dict(lr_device=P + 2),
                   dict(grad_norm=P + 1)):
        refused(g.moe_adamw_step, INVALID, base, **change)
    for bad in (dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(m_scale=None),
                dict(v_scale=None), dict(numel=-1), dict(param_dtype=2), dict(grad_dtype=-1),
                dict(master=None), dict(param_dtype=1), dict(param=P + 1), dict(grad=3 * P + 1),
                dict(master=2 * P + 2), dict(decay=-0.5), dict(decay=math.inf),
                dict(decay=math.nan)):
        refused(g.moe_adamw_step, INVALID, adamw_args(**bad))
    refused(g.moe_adamw_step, INVALID, dict(adamw_args(m=4 * P + 2), state_bits=32))


def test_adamw_moments_refuses():
    base = {k: v for k, v in adamw_args().items() if k in ("n", "tensors", "stream")}
    out = (ctypes.c_void_p * 1)(P)
    for change in (dict(m_out=None), dict(v_out=None), dict(m_out=(ctypes.c_void_p * 1)(None)),
                   dict(v_out=(ctypes.c_void_p * 1)(P + 1)), dict(n=-1),
                   dict(tensors=adamw_args(v_scale=None)["tensors"])):
        refused(g.moe_adamw_moments, INVALID, dict(base, m_out=out, v_out=out), **change)


def test_adamw_list_matches_the_header(tmp_path):
    src = tmp_path / "sz.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "moegmm.h"\n'
                   'int main(void) { printf("%zu %zu %zu\\n", sizeof(moe_adamw_tensor_t), '
                   'offsetof(moe_adamw_tensor_t, numel), offsetof(moe_adamw_tensor_t, decay));'
                   ' return 0; }\n')
    exe = tmp_path / "sz"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    size, numel, decay = map(int, subprocess.run([str(exe)], capture_output=True, text=True,
                                                 check=True).stdout.split())
    assert ctypes.sizeof(g.AdamWTensor) == size
    assert (g.AdamWTensor.numel.offset, g.AdamWTensor.decay.offset) == (numel, decay)


def test_permute_refuses():
    desc = g.make_desc(E=8, k=2, H=256, F=512, T_max=100)
    base = dict(desc=desc, T=4, topk_ids=P, topk_probs=P, x=P, counts=P, ws=P,
                ws_bytes=g.moe_workspace_size(desc), stream=0)
    for change in (dict(T=-1), dict(T=101), dict(topk_ids=None), dict(topk_probs=None),
                   dict(x=None), dict(counts=None), dict(ws=None), dict(x=P + 8), dict(ws=P + 16),
                   dict(topk_ids=P + 2), dict(topk_probs=P + 1), dict(counts=P + 2),
                   dict(desc=g.make_desc(E=0, k=2, H=256, F=512, T_max=100))):
        refused(g.moe_permute, INVALID, base, **change)
    refused(g.moe_permute, WORKSPACE, base, ws_bytes=64)


def test_nothing_to_do_returns_without_a_launch():
    n = g.moe_launch_count()
    g.moe_router_topk_fwd(**dict(TOPK, T=0, counts=None))
    g.moe_router_topk_bwd(P, 8, 1, P, P, 0, 8, 2, 1, 1, 1.0, None, 0, P, 8, 0)
    g.moe_residual_norm_fwd(**dict(FWD, M=0))
    g.moe_residual_norm_bwd(**dict(BWD, M=0, d_weight=None, d_post_weight=None))
    g.moe_adamw_moments(0, None, None, None, 0)
    assert g.moe_launch_count() == n


def test_names():
    assert g.SCORE == {"softmax": 0, "sigmoid": 1}
    assert len(g.KERNEL_NAMES) + len(g.MORE_KERNEL_NAMES) == 36
    assert g.MORE_KERNEL_NAMES[6] == "adamw"


def test_overlap():
    assert not g._overlap([(0, 8, True), (8, 16, True), (16, 16, True), (12, 12, False)])
    assert not g._overlap([(0, 8, False), (4, 12, False), (12, 16, True)])
    assert g._overlap([(0, 8, True), (4, 12, False)])
    assert g._overlap([(0, 8, False), (4, 6, True)])
    assert g._overlap([(0, 8, True), (0, 8, True)])


APART = dict(FWD, x=P, o=2 * P, x_new=3 * P, h=4 * P, post_weight=5 * P, gate=6 * P, weight=7 * P,
             rstd_post=8 * P, rstd=9 * P)
ROW = 64 * 2   # bytes of a row


@pytest.mark.parametrize("change", [
    dict(x_new=P + ROW), dict(x=3 * P + ROW), dict(x_new=P - ROW), dict(x_new=P + 16), dict(x_new=P + 3 * ROW),
    dict(x_new=2 * P + ROW), dict(h=P + ROW), dict(h=2 * P - ROW), dict(h=3 * P), dict(h=3 * P + ROW),
    dict(x_new=P + ROW, ldx=128, ldxn=64), dict(x_new=P + ROW - 16, ldx=128, ldxn=128),
    dict(x_new=P + 2 * ROW, ldx=128, ldxn=128), dict(x=P, x_dtype=1, x_new=2 * P),
    dict(M=1, x_new=P + 16), dict(M=1, x=3 * P + 16)])
def test_residual_norm_forward_refuses_shared_memory(change):
    refused(g.moe_residual_norm_fwd, INVALID, APART, **change)


BACK = dict(BWD, dh=P, dx_new=2 * P, x_new=3 * P, o=4 * P, dx=5 * P, d_o=6 * P, post_weight=7 * P,
            gate=8 * P, weight=9 * P, rstd_post=10 * P, rstd=11 * P, d_post_weight=12 * P,
            d_weight=13 * P, d_gate=14 * P, ws=15 * P)


@pytest.mark.parametrize("change", [
    dict(dx=2 * P + ROW), dict(dx=3 * P - ROW), dict(dx=P + 16), dict(dx=4 * P + ROW), dict(d_o=P + ROW),
    dict(d_o=4 * P - 16), dict(d_o=2 * P + ROW), dict(d_o=3 * P + ROW), dict(d_o=5 * P),
    dict(d_o=5 * P + ROW), dict(dx=P, x_dtype=1), dict(d_o=4 * P + ROW - 16, ldo=128, lddo=128)])
def test_residual_norm_backward_refuses_shared_memory(change):
    refused(g.moe_residual_norm_bwd, INVALID, BACK, **change)


@pytest.mark.parametrize("change", [
    dict(add_to=4 * P + 32, ld_add=8), dict(add_to=4 * P - 32, ld_add=8), dict(logits=4 * P + 64),
    dict(logits=4 * P, logits_dtype=0), dict(add_to=4 * P + 16, ld_add=16, ld_d=16)])
def test_router_topk_backward_refuses_shared_memory(change):
    base = dict(logits=P, ld_logits=8, logits_dtype=1, topk_ids=2 * P, d_weights=3 * P, T=4, E=8, k=2,
                score=0, renorm=0, scale=1.0, add_to=None, ld_add=0, d_logits=4 * P, ld_d=8, stream=0)
    refused(g.moe_router_topk_bwd, INVALID, base, **change)


# The same rows, columns of one wider matrix, neighbours: not refused. Without a GPU the launch fails.
IN_ORDER = [
    (g.moe_residual_norm_fwd, APART, [
        dict(), dict(x_new=P), dict(h=2 * P), dict(x_new=P, h=2 * P), dict(x_new=2 * P), dict(h=P),
        dict(x_new=P + 4 * ROW), dict(x_new=P + ROW, ldx=128, ldxn=128),
        dict(x=3 * P + ROW, ldx=128, ldxn=128), dict(x_new=P - ROW, ldx=128, ldxn=128),
        dict(M=1, x_new=P, ldxn=64, ldx=64), dict(M=1, x_new=P + ROW)]),
    (g.moe_residual_norm_bwd, BACK, [
        dict(), dict(dx=2 * P, d_o=P), dict(dx=2 * P, d_o=4 * P), dict(dx=3 * P),
        dict(d_o=5 * P + 4 * ROW), dict(d_o=4 * P + ROW, ldo=128, lddo=128)])]


@pytest.mark.parametrize("fn,base,change", [(f, b, c) for f, b, cs in IN_ORDER for c in cs])
def test_residual_norm_in_order(fn, base, change):
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are not memory")
    with pytest.raises(g.MoeError) as e:
        fn(**dict(base, **change))
    assert e.value.status not in (INVALID, UNSUPPORTED, WORKSPACE), str(e.value)
