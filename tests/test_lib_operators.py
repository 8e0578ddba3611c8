"""CPU-only checks of the operators around the expert layer: sizes of their workspaces and the
refusals of their host-side checks (none of these calls touches the device)."""
import ctypes
import math

import pytest

import grouped_gemm_device_gb300 as g
from grouped_gemm_device_gb300 import build as gbuild

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


ROUTER = dict(logits=P, ld_logits=8, topk_ids=P, token_mask=None, T=4, E=8, k=2, coef=0.01, loss=P,
              counts=P, mean_prob=P, n_valid=P, ws=P, ws_bytes=1 << 20, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(E=0), INVALID), (dict(E=257, ld_logits=257), INVALID), (dict(k=0), INVALID),
    (dict(k=9), INVALID), (dict(E=1, k=2), INVALID), (dict(T=-1), INVALID),
    (dict(ld_logits=7), INVALID), (dict(logits=None), INVALID), (dict(topk_ids=None), INVALID),
    (dict(loss=None), INVALID), (dict(counts=None), INVALID), (dict(ws=None), INVALID),
    (dict(n_valid=P + 2), INVALID), (dict(ws=P + 8), INVALID), (dict(ws_bytes=100), WORKSPACE)])
def test_router_loss_forward_refuses(change, status):
    refused(g.moe_router_loss_fwd, status, ROUTER, **change)


def test_router_loss_backward_refuses():
    base = dict(logits=P, ld_logits=8, topk_ids=P, topk_probs=P, d_probs=P, token_mask=None, T=4,
                E=8, k=2, coef=0.01, d_loss=None, counts=P, n_valid=P, d_logits=P, ld_d=8,
                stream=0)
    for change in (dict(topk_probs=None), dict(d_probs=None), dict(ld_d=7), dict(d_logits=None),
                   dict(counts=None), dict(n_valid=None), dict(k=0), dict(T=-1),
                   dict(d_logits=P + 1), dict(topk_ids=P + 2)):
        refused(g.moe_router_loss_bwd, INVALID, base, **change)


def test_router_loss_workspace():
    assert g.moe_router_loss_workspace(256) >= g.moe_router_loss_workspace(1) > 0
    for E in (0, 257, -3):
        with pytest.raises(g.MoeError):
            g.moe_router_loss_workspace(E)


LN = dict(x=P, ldx=64, gamma=P, beta=P, y=P, ldy=64, mean=P, rstd=P, M=4, N=64, eps=1e-5,
          x_dtype=0, w_dtype=0, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(ldx=63), INVALID), (dict(ldy=63), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID), (dict(x=None), INVALID),
    (dict(y=None), INVALID), (dict(x_dtype=2), INVALID), (dict(w_dtype=-1), INVALID),
    (dict(x_dtype=1, w_dtype=0), UNSUPPORTED), (dict(x=P + 1), INVALID),
    (dict(gamma=P + 1), INVALID), (dict(mean=P + 2), INVALID),
    (dict(N=1 << 31, ldx=1 << 31, ldy=1 << 31), UNSUPPORTED)])
def test_layernorm_forward_refuses(change, status):
    refused(g.moe_layernorm_fwd, status, LN, **change)


def test_layernorm_backward_refuses():
    base = dict(dy=P, lddy=64, x=P, ldx=64, gamma=P, mean=P, rstd=P, dx=P, lddx=64, dgamma=P,
                dbeta=P, M=4, N=64, x_dtype=0, w_dtype=1, ws=P, ws_bytes=1 << 20, stream=0)
    for change in (dict(dy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=None),
                   dict(lddy=63), dict(lddx=1), dict(ws=None), dict(ws=P + 4),
                   dict(dgamma=P + 2), dict(N=0)):
        refused(g.moe_layernorm_bwd, INVALID, base, **change)
    refused(g.moe_layernorm_bwd, WORKSPACE, base, ws_bytes=g.moe_layernorm_workspace(4, 64) - 1)
    refused(g.moe_layernorm_bwd, UNSUPPORTED, base, x_dtype=1, w_dtype=0)


def test_layernorm_workspace_grows_with_its_arguments():
    a, b, c = (g.moe_layernorm_workspace(*s) for s in ((1, 64), (100, 64), (100, 128)))
    assert 0 < a <= b <= c and g.moe_layernorm_workspace(0, 1) > 0
    with pytest.raises(g.MoeError):
        g.moe_layernorm_workspace(1, 0)


def clip_args(ptrs=(P, P), outs=None, numel=(4, 4), types=(0, 1)):
    n = len(ptrs)
    return dict(n=n, grads=(ctypes.c_void_p * n)(*ptrs),
                outs=None if outs is None else (ctypes.c_void_p * n)(*outs),
                numel=(ctypes.c_int64 * n)(*numel), dtypes=(ctypes.c_int32 * n)(*types),
                max_norm=1.0, norm=P, ws=P, ws_bytes=g.moe_grad_clip_workspace(), stream=0)


def test_grad_clip_refuses():
    base = clip_args()
    for change in (dict(n=-1), dict(n=65537), dict(grads=None), dict(numel=None),
                   dict(dtypes=None), dict(max_norm=0.0), dict(max_norm=-1.0),
                   dict(max_norm=math.nan), dict(norm=None), dict(ws=None), dict(ws=P + 8),
                   dict(norm=P + 2)):
        refused(g.moe_grad_clip, INVALID, base, **change)
    refused(g.moe_grad_clip, WORKSPACE, base, ws_bytes=8)
    for bad in (clip_args(ptrs=(P, None)), clip_args(ptrs=(P + 1, P)), clip_args(ptrs=(P, P + 2)),
                clip_args(numel=(4, -1)), clip_args(types=(0, 2)), clip_args(outs=(P, None)),
                clip_args(outs=(P + 1, P)), dict(clip_args(outs=(P, P)), max_norm=math.inf)):
        refused(g.moe_grad_clip, INVALID, bad)


ROWS = dict(x=P, ldx=256, M=4, N=256, q_row=P, ld_qrow=256, s_row=P, ld_srow=4, q_col=P, ld_qcol=16,
            s_col=P, ld_scol=256, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(ldx=255), INVALID),
    (dict(ld_qrow=255), INVALID), (dict(ld_srow=3), INVALID), (dict(ld_qcol=3), INVALID),
    (dict(ld_scol=255), INVALID), (dict(s_row=None), INVALID), (dict(q_col=None), INVALID),
    (dict(q_row=None, s_row=None, q_col=None, s_col=None), INVALID), (dict(x=None), INVALID),
    (dict(x=P + 1), INVALID), (dict(s_row=P + 2), INVALID),
    (dict(M=1 << 31, ld_srow=1 << 31, ld_qcol=1 << 31), UNSUPPORTED)])
def test_fp8_quantize_rows_refuses(change, status):
    refused(g.fp8_block_quantize_rows, status, ROWS, **change)


def test_fp8_quantize_weight_refuses():
    base = dict(w=P, ldw=256, N=64, K=256, q=P, ldq=256, s=P, qt=P, ldqt=64, st=P, stream=0)
    for change in (dict(N=-1), dict(w=None), dict(q=None), dict(s=None), dict(qt=None),
                   dict(st=None), dict(ldw=255), dict(ldq=255), dict(ldqt=63), dict(w=P + 1),
                   dict(s=P + 1)):
        refused(g.fp8_block_quantize_weight, INVALID, base, **change)


GEMM = dict(a=P, lda=256, sa=P, ld_sa=8, b=P, ldb=256, sb=P, ld_sb=2, b_scale=1, c=P, ldc=64,
            c_dtype=0, M=8, N=64, K=256, err=None, stream=0)


@pytest.mark.parametrize("change,status", [
    (dict(M=-1), INVALID), (dict(K=0), INVALID), (dict(lda=255), INVALID), (dict(lda=264), INVALID),
    (dict(ldb=240), INVALID), (dict(ldc=63), INVALID), (dict(ld_sa=4), INVALID),
    (dict(ld_sa=10), INVALID), (dict(ld_sb=1), INVALID), (dict(b_scale=2), INVALID),
    (dict(b_scale=0, ld_sb=63), INVALID), (dict(b_scale=0, ld_sb=66), INVALID),
    (dict(b_scale=0, ld_sb=64, sb=P + 4), INVALID), (dict(a=P + 8), INVALID),
    (dict(b=P + 8), INVALID), (dict(sa=P + 4), INVALID), (dict(sb=P + 2), INVALID),
    (dict(c=P + 1), INVALID), (dict(c=P + 2, c_dtype=1), INVALID), (dict(c_dtype=2), INVALID),
    (dict(a=None), INVALID), (dict(b=None), INVALID), (dict(sa=None), INVALID),
    (dict(sb=None), INVALID), (dict(c=None), INVALID), (dict(err=P + 2), INVALID),
    (dict(M=(1 << 31) - 1, ld_sa=1 << 31), UNSUPPORTED)])
def test_fp8_gemm_refuses(change, status):
    refused(g.fp8_block_gemm, status, GEMM, **change)


def test_nothing_to_do_returns_without_a_launch():
    n = g.moe_launch_count()
    g.moe_layernorm_fwd(**dict(LN, M=0))
    g.fp8_block_quantize_rows(**dict(ROWS, M=0))
    g.fp8_block_gemm(**dict(GEMM, M=0))
    g.fp8_block_gemm(**dict(GEMM, N=0))
    assert g.moe_launch_count() == n


def test_dtype_names_match_the_header():
    assert g.DTYPE == {"bf16": 0, "fp32": 1}
    assert g.KERNEL_NAMES[19] == "router_loss" and g.KERNEL_NAMES[27] == "fp8_gemm"
    assert len(g.KERNEL_NAMES) == 28


def test_calls_refuse_wrong_arguments(lib):
    """The classes' own way into the library (csrc/calls.c): counts and conversions of arguments;
    statuses come back as numbers."""
    calls = g._load_calls()
    assert calls.moe_grad_clip(-1, 0, None, 0, 0, 1.0, None, None, 0, None) == 1
    for args in ((), (0,) * 9, (0,) * 11):
        with pytest.raises(TypeError):
            calls.moe_grad_clip(*args)
    with pytest.raises(TypeError):
        calls.moe_grad_clip("0", 0, None, 0, 0, 1.0, None, None, 0, None)
    with pytest.raises(OverflowError):
        calls.moe_grad_clip(1 << 31, 0, None, 0, 0, 1.0, None, None, 0, None)
    with pytest.raises(TypeError):
        calls.bind(0)
