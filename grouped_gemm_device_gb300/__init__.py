"""Python binding of libmoegmm (the GB300 fused grouped expert MLP).

Argument marshalling only: every step of the layer runs in the library's CUDA kernels. The
functions below carry the C ABI's names (include/moegmm.h) and accept torch tensors (their
device pointers are passed) or raw integer addresses. `MoELayer` is plumbing on top: it
allocates the caller-owned buffers with torch and calls the same entry points.

There is no fallback: if the shared library is missing, `load()` raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import importlib.machinery
import importlib.util
import math
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libmoegmm.so")
CALLS_PATH = os.path.join(_PKG, "_lib", "_moecalls.so")

PREC = {"bf16": 0, "mxfp8": 1, "nvfp4": 2}
ACT = {"swiglu": 0, "clamped_swiglu": 1, "geglu": 2, "srelu": 3}
EXTRA_BIAS, EXTRA_SCALE = 1, 2  # moe_layer_desc_t.extras bits
DTYPE = {"bf16": 0, "fp32": 1}  # moe_dtype_t
SCORE = {"softmax": 0, "sigmoid": 1}  # moe_score_t
DEVERR = {0: "none", 1: "capacity", 2: "timeout", 3: "bad_id"}

KERNEL_NAMES = ("route_topk", "assign_rows", "gather_x", "gemm_fc1_fprop", "gemm_fc2_fprop",
                "combine_y", "gather_dy", "gemm_fc2_dgrad", "dprob_reduce", "gemm_fc2_wgrad",
                "gemm_fc1_dgrad", "combine_dx", "gemm_fc1_wgrad", "mxfp8_quantize", "pack_fc1",
                "extras_reduce", "nvfp4_amax", "nvfp4_quantize", "route_export", "router_loss",
                "router_grad", "layernorm_fwd", "layernorm_bwd", "layernorm_reduce", "grad_norm",
                "grad_scale", "fp8_quantize", "fp8_gemm")
MORE_KERNEL_NAMES = ("count_ids", "router_topk", "router_topk_grad", "residual_norm_fwd",
                     "residual_norm_bwd", "residual_norm_reduce", "adamw", "adamw_moments")
# moe_ws_layout_t.nv_amax slots (fp32 [16], first 10 used)
NV_AMAX = ("x", "xt", "w1", "w2", "a", "at", "dy", "dyt", "dz", "dzt")

EXPORTS = ("moe_timeline_begin", "moe_timeline_end", "moe_workspace_size", "moe_workspace_layout", "moe_route_permute",
           "moe_grouped_mlp_fwd", "moe_grouped_mlp_bwd", "mxfp8_quantize", "moe_pack_fc1_weight",
           "moe_get_error", "moe_clear_error", "moe_gemm_ctas", "moe_launch_count",
           "moe_last_error_string", "moe_selftest_wait_timeout", "moe_selftest_gemm_timeout",
           "moe_route_export",
           "moe_grouped_mlp_fwd_ex",
           "moe_grouped_mlp_bwd_ex", "nvfp4_amax", "nvfp4_quantize",
           "moe_router_loss_workspace", "moe_router_loss_fwd", "moe_router_loss_bwd",
           "moe_layernorm_fwd", "moe_layernorm_workspace", "moe_layernorm_bwd",
           "moe_grad_clip_workspace", "moe_grad_clip", "fp8_block_quantize_rows",
           "fp8_block_quantize_weight", "fp8_block_gemm", "moe_permute", "moe_router_topk_fwd",
           "moe_router_topk_bwd", "moe_residual_norm_fwd", "moe_residual_norm_workspace",
           "moe_residual_norm_bwd", "moe_adamw_step", "moe_adamw_moments")


class LayerDesc(ctypes.Structure):
    _fields_ = [("E", ctypes.c_int32), ("k", ctypes.c_int32), ("H", ctypes.c_int32),
                ("F", ctypes.c_int32), ("T_max", ctypes.c_int32), ("precision", ctypes.c_int32),
                ("activation", ctypes.c_int32), ("beta", ctypes.c_float),
                ("gate_max", ctypes.c_float), ("lin_lo", ctypes.c_float),
                ("lin_hi", ctypes.c_float), ("lin_offset", ctypes.c_float),
                ("sm_margin", ctypes.c_int32), ("ilv", ctypes.c_int32), ("align", ctypes.c_int32),
                ("recompute", ctypes.c_int32), ("extras", ctypes.c_int32),
                ("rht_mask", ctypes.c_uint32), ("reuse_weights", ctypes.c_int32),
                ("pdl", ctypes.c_int32)]


class WsLayout(ctypes.Structure):
    _fields_ = [("total", ctypes.c_size_t), ("R_cap", ctypes.c_int64), ("err", ctypes.c_size_t),
                ("offsets", ctypes.c_size_t), ("row_of", ctypes.c_size_t),
                ("src_of", ctypes.c_size_t), ("row_prob", ctypes.c_size_t),
                ("x_perm", ctypes.c_size_t), ("z", ctypes.c_size_t), ("a_s", ctypes.c_size_t),
                ("y_perm", ctypes.c_size_t), ("dy_perm", ctypes.c_size_t),
                ("dz", ctypes.c_size_t), ("dx_perm", ctypes.c_size_t),
                ("dprob_part", ctypes.c_size_t), ("ext_part", ctypes.c_size_t),
                ("mx_base", ctypes.c_size_t), ("nv_amax", ctypes.c_size_t),
                ("nv_base", ctypes.c_size_t)]


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor_t"""
    _fields_ = [("param", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("numel", ctypes.c_int64), ("param_dtype", ctypes.c_int32),
                ("grad_dtype", ctypes.c_int32), ("decay", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F32 = ctypes.c_float
_F64 = ctypes.c_double
_DP = ctypes.POINTER(LayerDesc)


def load():
    """Load the shared library (build it first with __graft_entry__.build() or
    `python -m grouped_gemm_device_gb300.build`). Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libmoegmm.so not built ({LIB_PATH}); run the build step first")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "moe_workspace_size": (_SZ, [_DP]),
        "moe_workspace_layout": (_I32, [_DP, ctypes.POINTER(WsLayout)]),
        "moe_route_permute": (_I32, [_DP, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "moe_grouped_mlp_fwd": (_I32, [_DP, _I32, _P, _P, _P, _P, _SZ, _P]),
        "moe_grouped_mlp_bwd": (_I32, [_DP, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "mxfp8_quantize": (_I32, [_P, _I64, _I64, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P]),
        "nvfp4_amax": (_I32, [_P, _I64, _I64, ctypes.c_uint32, _P, _P, _P]),
        "nvfp4_quantize": (_I32, [_P, _I64, _I64, _P, _P, _I32, ctypes.c_uint32, _P, _P, _P, _P,
                                  _P]),
        "moe_pack_fc1_weight": (_I32, [_P, _P, _I32, _I32, _I32, _I32, _I32, _I32, _P]),
        "moe_get_error": (_I32, [_DP, _P, ctypes.POINTER(_I32), _P]),
        "moe_clear_error": (_I32, [_DP, _P, _P]),
        "moe_gemm_ctas": (_I32, [_DP]),
        "moe_launch_count": (ctypes.c_uint64, []),
        "moe_last_error_string": (ctypes.c_char_p, []),
        "moe_timeline_begin": (_I32, [ctypes.POINTER(_P), _I32]),
        "moe_timeline_end": (_I32, [ctypes.POINTER(_I32)]),
        "moe_route_permute_noalloc": (_I32, [_DP, _I32, _P, _P, _P, _P, _P, _P, _P, _I64, _P]),
        "moe_selftest_wait_timeout": (_I32, [_P, ctypes.c_uint64, _P]),
        "moe_selftest_gemm_timeout": (_I32, [_DP, _P, _SZ, _P, ctypes.c_uint64, _P]),
        "moe_route_export": (_I32, [_DP, _P, _SZ, _I32, _P, _P, _P, _P, _P]),
        "moe_grouped_mlp_fwd_ex": (_I32, [_DP, _I32, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        "moe_grouped_mlp_bwd_ex": (_I32, [_DP, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                          _SZ, _P]),
        "moe_router_loss_workspace": (_SZ, [_I32]),
        "moe_router_loss_fwd": (_I32, [_P, _I64, _P, _P, _I32, _I32, _I32, _F32, _P, _P, _P, _P,
                                       _P, _SZ, _P]),
        "moe_router_loss_bwd": (_I32, [_P, _I64, _P, _P, _P, _P, _I32, _I32, _I32, _F32, _P, _P,
                                       _P, _P, _I64, _P]),
        "moe_layernorm_fwd": (_I32, [_P, _I64, _P, _P, _P, _I64, _P, _P, _I64, _I64, _F32, _I32,
                                     _I32, _P]),
        "moe_layernorm_workspace": (_SZ, [_I64, _I64]),
        "moe_layernorm_bwd": (_I32, [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _P, _I64, _I64,
                                     _I32, _I32, _P, _SZ, _P]),
        "moe_grad_clip_workspace": (_SZ, []),
        "moe_grad_clip": (_I32, [_I32, _P, _P, _P, _P, _F32, _P, _P, _SZ, _P]),
        "fp8_block_quantize_rows": (_I32, [_P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I64, _P,
                                           _I64, _P]),
        "fp8_block_quantize_weight": (_I32, [_P, _I64, _I64, _I64, _P, _I64, _P, _P, _I64, _P,
                                             _P]),
        "fp8_block_gemm": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _I32, _P, _I64, _I32,
                                  _I64, _I64, _I64, _P, _P]),
        "moe_permute": (_I32, [_DP, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
        "moe_router_topk_fwd": (_I32, [_P, _I64, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32, _I32,
                                       _I32, _I32, _F32, _P, _P, _P, _P]),
        "moe_router_topk_bwd": (_I32, [_P, _I64, _I32, _P, _P, _I32, _I32, _I32, _I32, _I32, _F32,
                                       _P, _I64, _P, _I64, _P]),
        "moe_residual_norm_fwd": (_I32, [_P, _I64, _P, _I64, _P, _P, _P, _P, _I64, _P, _I64, _P,
                                         _P, _I64, _I64, _F32, _I32, _F32, _I32, _I32, _I32, _P]),
        "moe_residual_norm_workspace": (_SZ, [_I64, _I64]),
        "moe_residual_norm_bwd": (_I32, [_P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _P, _P, _P,
                                         _P, _P, _I64, _P, _I64, _P, _P, _P, _I64, _I64, _F32,
                                         _I32, _I32, _I32, _I32, _P, _SZ, _P]),
        "moe_adamw_step": (_I32, [_I32, _P, _I32, _F64, _P, _F64, _F64, _F64, _P, _F32,
                                  ctypes.c_uint64, _P, _P]),
        "moe_adamw_moments": (_I32, [_I32, _P, _P, _P, _P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


# Functions of the library that the operator classes call through csrc/calls.c, in the order of its
# bind(): the same arguments as above, without ctypes' time.
_CALLS = ("moe_router_loss_fwd", "moe_router_loss_bwd", "moe_layernorm_fwd", "moe_layernorm_bwd",
          "moe_grad_clip", "fp8_block_quantize_rows", "fp8_block_quantize_weight",
          "fp8_block_gemm", "moe_router_topk_fwd", "moe_router_topk_bwd", "moe_residual_norm_fwd",
          "moe_residual_norm_bwd", "moe_adamw_step", "moe_adamw_moments")
_calls = None


def _load_calls():
    """The module of csrc/calls.c, bound to the library. Raises if it is missing."""
    global _calls
    if _calls is None:
        lib = load()
        if not os.path.exists(CALLS_PATH):
            raise RuntimeError(f"{CALLS_PATH} not built; run the build step first")
        spec = importlib.util.spec_from_file_location(
            "_moecalls", CALLS_PATH,
            loader=importlib.machinery.ExtensionFileLoader("_moecalls", CALLS_PATH))
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        mod.bind(*[ctypes.cast(getattr(lib, name), _P).value for name in _CALLS])
        _calls = mod
    return _calls


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"status {status}: {msg}")
        self.status = status


def _check(st: int):
    if st != 0:
        raise MoeError(st, load().moe_last_error_string().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_cuda = None  # torch._C once CUDA is initialised


def _stream(stream) -> int | None:
    global _cuda
    if stream is None:
        if _cuda is None:
            import torch
            if not torch.cuda.is_initialized():
                return torch.cuda.current_stream().cuda_stream
            _cuda = torch._C
        # the current stream's handle without building a Stream object
        return _cuda._cuda_getCurrentRawStream(_cuda._cuda_getDevice())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_desc(E, k, H, F, T_max, precision="bf16", activation="swiglu", beta=1.0,
              gate_max=math.inf, lin_lo=-math.inf, lin_hi=math.inf, lin_offset=0.0,
              sm_margin=0, ilv=64, align=32, recompute=False, extras=0,
              rht_mask=0, reuse_weights=False, pdl=False) -> LayerDesc:
    """extras: bit 0 FC1 bias, bit 1 feature scale (EXTRA_BIAS | EXTRA_SCALE). rht_mask: the
    16 signs of the NVFP4 weight-gradient rotation (bit j set: row j of a block negated).
    reuse_weights: the forward reuses the workspace's block-scaled weight copies. pdl: launch
    the call's kernels with programmatic stream serialization."""
    return LayerDesc(E, k, H, F, T_max, PREC[precision], ACT[activation], beta, gate_max,
                     lin_lo, lin_hi, lin_offset, sm_margin, ilv, align, int(recompute),
                     int(extras), int(rht_mask) & 0xFFFF, int(reuse_weights), int(pdl))


def desc_from_config(cfg, T_max=None, sm_margin=0, recompute=False, extras=0,
                     rht_mask=None) -> LayerDesc:
    """A description of a synthetic workload (synth.LayerConfig); an NVFP4 layer takes the
    workload's seeded rotation signs unless rht_mask is given."""
    if rht_mask is None:
        from . import synth
        rht_mask = synth.gen_rht_mask(cfg) if cfg.precision == "nvfp4" else 0
    return make_desc(cfg.E, cfg.k, cfg.H, cfg.F, cfg.T if T_max is None else T_max,
                     cfg.precision, cfg.activation, cfg.beta, cfg.gate_max, cfg.lin_lo,
                     cfg.lin_hi, cfg.lin_offset, sm_margin, cfg.ilv, cfg.align, recompute,
                     extras, rht_mask)


# ------------------------------------------------------------------ C ABI, same names
def moe_workspace_size(desc: LayerDesc) -> int:
    n = load().moe_workspace_size(ctypes.byref(desc))
    if n == 0:
        raise MoeError(1, load().moe_last_error_string().decode())
    return n


def moe_workspace_layout(desc: LayerDesc) -> WsLayout:
    out = WsLayout()
    _check(load().moe_workspace_layout(ctypes.byref(desc), ctypes.byref(out)))
    return out


def moe_route_permute(desc, T, logits, x, topk_ids, topk_probs, counts, ws, ws_bytes,
                      stream=None):
    _check(load().moe_route_permute(ctypes.byref(desc), T, _ptr(logits), _ptr(x), _ptr(topk_ids),
                                    _ptr(topk_probs), _ptr(counts), _ptr(ws), ws_bytes,
                                    _stream(stream)))


def moe_route_permute_noalloc(desc, T, logits, x, topk_ids, topk_probs, counts, offsets,
                              x_perm, x_perm_rows, stream=None):
    """Route + permute into caller buffers with no workspace and no device allocation (the
    library keeps its small scratch in a static device array; see include/moegmm.h)."""
    _check(load().moe_route_permute_noalloc(ctypes.byref(desc), T, _ptr(logits), _ptr(x),
                                            _ptr(topk_ids), _ptr(topk_probs), _ptr(counts),
                                            _ptr(offsets), _ptr(x_perm), x_perm_rows,
                                            _stream(stream)))


def moe_grouped_mlp_fwd(desc, T, w1_packed, w2, y, ws, ws_bytes, stream=None):
    _check(load().moe_grouped_mlp_fwd(ctypes.byref(desc), T, _ptr(w1_packed), _ptr(w2), _ptr(y),
                                      _ptr(ws), ws_bytes, _stream(stream)))


def moe_grouped_mlp_bwd(desc, T, dy, w1_packed, w2, dx, dw1_packed, dw2, d_probs, ws, ws_bytes,
                        stream=None):
    _check(load().moe_grouped_mlp_bwd(ctypes.byref(desc), T, _ptr(dy), _ptr(w1_packed), _ptr(w2),
                                      _ptr(dx), _ptr(dw1_packed), _ptr(dw2), _ptr(d_probs),
                                      _ptr(ws), ws_bytes, _stream(stream)))


def moe_grouped_mlp_fwd_ex(desc, T, w1_packed, w2, fc1_bias, feat_scale, y, ws, ws_bytes,
                           stream=None):
    _check(load().moe_grouped_mlp_fwd_ex(ctypes.byref(desc), T, _ptr(w1_packed), _ptr(w2),
                                         _ptr(fc1_bias), _ptr(feat_scale), _ptr(y), _ptr(ws),
                                         ws_bytes, _stream(stream)))


def moe_grouped_mlp_bwd_ex(desc, T, dy, w1_packed, w2, feat_scale, dx, dw1_packed, dw2, d_probs,
                           d_fc1_bias, d_feat_scale, ws, ws_bytes, stream=None):
    _check(load().moe_grouped_mlp_bwd_ex(ctypes.byref(desc), T, _ptr(dy), _ptr(w1_packed),
                                         _ptr(w2), _ptr(feat_scale), _ptr(dx), _ptr(dw1_packed),
                                         _ptr(dw2), _ptr(d_probs), _ptr(d_fc1_bias),
                                         _ptr(d_feat_scale), _ptr(ws), ws_bytes, _stream(stream)))


def mxfp8_quantize(inp, M, N, rowwise, colwise, q_row=None, s_row=None, q_col=None, s_col=None,
                   stream=None, group_offsets=None, num_groups=0):
    """group_offsets: int32 device tensor [num_groups + 1]; column-wise blocks then restart at
    each group's first row and s_col is [N, mxfp8_grouped_scale_cols(M, num_groups)]."""
    _check(load().mxfp8_quantize(_ptr(inp), M, N, int(rowwise), int(colwise),
                                 _ptr(group_offsets), int(num_groups), _ptr(q_row), _ptr(s_row),
                                 _ptr(q_col), _ptr(s_col), _stream(stream)))


def mxfp8_grouped_scale_cols(M, num_groups) -> int:
    """Entries per column of the grouped column-wise scales (include/moegmm.h)."""
    return 4 * ((-(-M // 32) + num_groups + 3) // 4)


def nvfp4_amax(inp, M, N, sign_mask, amax, amax_rht=None, stream=None):
    _check(load().nvfp4_amax(_ptr(inp), M, N, int(sign_mask) & 0xFFFF, _ptr(amax),
                             _ptr(amax_rht), _stream(stream)))


def nvfp4_quantize(inp, M, N, amax_row, amax_col, rht, sign_mask, q_row=None, s_row=None,
                   q_col=None, s_col=None, stream=None):
    _check(load().nvfp4_quantize(_ptr(inp), M, N, _ptr(amax_row), _ptr(amax_col), int(rht),
                                 int(sign_mask) & 0xFFFF, _ptr(q_row), _ptr(s_row), _ptr(q_col),
                                 _ptr(s_col), _stream(stream)))


def moe_pack_fc1_weight(src, dst, E, H, F, gated, ilv, inverse, stream=None):
    _check(load().moe_pack_fc1_weight(_ptr(src), _ptr(dst), E, H, F, int(gated), ilv,
                                      int(inverse), _stream(stream)))


def moe_selftest_wait_timeout(err, limit_ns, stream=None):
    """Enqueue the bounded-wait self-test: a wait nothing completes gives up after limit_ns
    and writes the timeout code into the device int32 `err`."""
    _check(load().moe_selftest_wait_timeout(_ptr(err), int(limit_ns), _stream(stream)))


def moe_selftest_gemm_timeout(desc, ws, ws_bytes, w2, limit_ns, stream=None):
    """Enqueue the FC2 forward GEMM of a routed BF16 layer with its loads withheld: every wait
    of the kernel runs out after limit_ns and the workspace error word records the timeout."""
    _check(load().moe_selftest_gemm_timeout(ctypes.byref(desc), _ptr(ws), ws_bytes, _ptr(w2),
                                            int(limit_ns), _stream(stream)))


def moe_route_export(desc, ws, ws_bytes, T, offsets=None, row_of=None, src_of=None,
                     row_prob=None, stream=None):
    """Copy the routing maps of the last route on ws into caller tensors (any may be None)."""
    _check(load().moe_route_export(ctypes.byref(desc), _ptr(ws), ws_bytes, int(T),
                                   _ptr(offsets), _ptr(row_of), _ptr(src_of), _ptr(row_prob),
                                   _stream(stream)))


def moe_permute(desc, T, topk_ids, topk_probs, x, counts, ws, ws_bytes, stream=None):
    """Permute by given ids and weights (ids outside [0, E): dropped slots)."""
    _check(load().moe_permute(ctypes.byref(desc), T, _ptr(topk_ids), _ptr(topk_probs), _ptr(x),
                              _ptr(counts), _ptr(ws), ws_bytes, _stream(stream)))


def moe_router_topk_fwd(logits, ld_logits, logits_dtype, bias, token_mask, T, E, k, score, n_group,
                        topk_group, group_top, renorm, scale, topk_ids, topk_weights, counts,
                        stream=None):
    """logits_dtype: a value of DTYPE, score: one of SCORE."""
    _check(load().moe_router_topk_fwd(_ptr(logits), ld_logits, logits_dtype, _ptr(bias),
                                      _ptr(token_mask), T, E, k, score, n_group, topk_group,
                                      group_top, int(renorm), scale, _ptr(topk_ids),
                                      _ptr(topk_weights), _ptr(counts), _stream(stream)))


def moe_router_topk_bwd(logits, ld_logits, logits_dtype, topk_ids, d_weights, T, E, k, score,
                        renorm, scale, add_to, ld_add, d_logits, ld_d, stream=None):
    _check(load().moe_router_topk_bwd(_ptr(logits), ld_logits, logits_dtype, _ptr(topk_ids),
                                      _ptr(d_weights), T, E, k, score, int(renorm), scale,
                                      _ptr(add_to), ld_add, _ptr(d_logits), ld_d,
                                      _stream(stream)))


def moe_router_loss_workspace(E) -> int:
    n = load().moe_router_loss_workspace(E)
    if n == 0:
        raise MoeError(1, load().moe_last_error_string().decode())
    return n


def moe_router_loss_fwd(logits, ld_logits, topk_ids, token_mask, T, E, k, coef, loss, counts,
                        mean_prob, n_valid, ws, ws_bytes, stream=None):
    _check(load().moe_router_loss_fwd(_ptr(logits), ld_logits, _ptr(topk_ids), _ptr(token_mask), T,
                                      E, k, coef, _ptr(loss), _ptr(counts), _ptr(mean_prob),
                                      _ptr(n_valid), _ptr(ws), ws_bytes, _stream(stream)))


def moe_router_loss_bwd(logits, ld_logits, topk_ids, topk_probs, d_probs, token_mask, T, E, k,
                        coef, d_loss, counts, n_valid, d_logits, ld_d, stream=None):
    _check(load().moe_router_loss_bwd(_ptr(logits), ld_logits, _ptr(topk_ids), _ptr(topk_probs),
                                      _ptr(d_probs), _ptr(token_mask), T, E, k, coef,
                                      _ptr(d_loss), _ptr(counts), _ptr(n_valid), _ptr(d_logits),
                                      ld_d, _stream(stream)))


def moe_layernorm_fwd(x, ldx, gamma, beta, y, ldy, mean, rstd, M, N, eps, x_dtype, w_dtype,
                      stream=None):
    """x_dtype, w_dtype: values of DTYPE."""
    _check(load().moe_layernorm_fwd(_ptr(x), ldx, _ptr(gamma), _ptr(beta), _ptr(y), ldy,
                                    _ptr(mean), _ptr(rstd), M, N, eps, x_dtype, w_dtype,
                                    _stream(stream)))


def moe_layernorm_workspace(M, N) -> int:
    n = load().moe_layernorm_workspace(M, N)
    if n == 0:
        raise MoeError(1, load().moe_last_error_string().decode())
    return n


def moe_layernorm_bwd(dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx, dgamma, dbeta, M, N, x_dtype,
                      w_dtype, ws, ws_bytes, stream=None):
    _check(load().moe_layernorm_bwd(_ptr(dy), lddy, _ptr(x), ldx, _ptr(gamma), _ptr(mean),
                                    _ptr(rstd), _ptr(dx), lddx, _ptr(dgamma), _ptr(dbeta), M, N,
                                    x_dtype, w_dtype, _ptr(ws), ws_bytes, _stream(stream)))


def moe_residual_norm_fwd(x, ldx, o, ldo, post_weight, gate, weight, x_new, ldxn, h, ldh,
                          rstd_post, rstd, M, N, scale, post_norm, eps, x_dtype, o_dtype, w_dtype,
                          stream=None):
    """x_dtype, o_dtype, w_dtype: values of DTYPE."""
    _check(load().moe_residual_norm_fwd(_ptr(x), ldx, _ptr(o), ldo, _ptr(post_weight), _ptr(gate),
                                        _ptr(weight), _ptr(x_new), ldxn, _ptr(h), ldh,
                                        _ptr(rstd_post), _ptr(rstd), M, N, scale, int(post_norm),
                                        eps, x_dtype, o_dtype, w_dtype, _stream(stream)))


def moe_residual_norm_workspace(M, N) -> int:
    n = load().moe_residual_norm_workspace(M, N)
    if n == 0:
        raise MoeError(1, load().moe_last_error_string().decode())
    return n


def moe_residual_norm_bwd(dh, lddh, dx_new, lddxn, x_new, ldxn, o, ldo, post_weight, gate, weight,
                          rstd_post, rstd, dx, lddx, d_o, lddo, d_post_weight, d_weight, d_gate, M,
                          N, scale, post_norm, x_dtype, o_dtype, w_dtype, ws, ws_bytes,
                          stream=None):
    _check(load().moe_residual_norm_bwd(_ptr(dh), lddh, _ptr(dx_new), lddxn, _ptr(x_new), ldxn,
                                        _ptr(o), ldo, _ptr(post_weight), _ptr(gate), _ptr(weight),
                                        _ptr(rstd_post), _ptr(rstd), _ptr(dx), lddx, _ptr(d_o),
                                        lddo, _ptr(d_post_weight), _ptr(d_weight), _ptr(d_gate), M,
                                        N, scale, int(post_norm), x_dtype, o_dtype, w_dtype,
                                        _ptr(ws), ws_bytes, _stream(stream)))


def moe_adamw_step(n, tensors, state_bits, lr, lr_device, beta1, beta2, eps, grad_norm, max_norm,
                   seed, counters, stream=None):
    """tensors: a ctypes array of AdamWTensor in host memory (include/moegmm.h)."""
    _check(load().moe_adamw_step(n, tensors, state_bits, lr, _ptr(lr_device), beta1, beta2, eps,
                                 _ptr(grad_norm), max_norm, seed, _ptr(counters),
                                 _stream(stream)))


def moe_adamw_moments(n, tensors, m_out, v_out, stream=None):
    """m_out, v_out: ctypes arrays of addresses in host memory."""
    _check(load().moe_adamw_moments(n, tensors, m_out, v_out, _stream(stream)))


def moe_grad_clip_workspace() -> int:
    return load().moe_grad_clip_workspace()


def moe_grad_clip(n, grads, outs, numel, dtypes, max_norm, norm, ws, ws_bytes, stream=None):
    """grads, outs (or None), numel, dtypes: ctypes arrays in host memory (include/moegmm.h)."""
    _check(load().moe_grad_clip(n, grads, outs, numel, dtypes, max_norm, _ptr(norm), _ptr(ws),
                                ws_bytes, _stream(stream)))


def fp8_block_quantize_rows(x, ldx, M, N, q_row=None, ld_qrow=0, s_row=None, ld_srow=0, q_col=None,
                            ld_qcol=0, s_col=None, ld_scol=0, stream=None):
    _check(load().fp8_block_quantize_rows(_ptr(x), ldx, M, N, _ptr(q_row), ld_qrow, _ptr(s_row),
                                          ld_srow, _ptr(q_col), ld_qcol, _ptr(s_col), ld_scol,
                                          _stream(stream)))


def fp8_block_quantize_weight(w, ldw, N, K, q, ldq, s, qt=None, ldqt=0, st=None, stream=None):
    _check(load().fp8_block_quantize_weight(_ptr(w), ldw, N, K, _ptr(q), ldq, _ptr(s), _ptr(qt),
                                            ldqt, _ptr(st), _stream(stream)))


def fp8_block_gemm(a, lda, sa, ld_sa, b, ldb, sb, ld_sb, b_scale, c, ldc, c_dtype, M, N, K,
                   err=None, stream=None):
    """b_scale: 1 for 128 x 128 blocks of b, 0 for 1 x 128; c_dtype: a value of DTYPE."""
    _check(load().fp8_block_gemm(_ptr(a), lda, _ptr(sa), ld_sa, _ptr(b), ldb, _ptr(sb), ld_sb,
                                 b_scale, _ptr(c), ldc, c_dtype, M, N, K, _ptr(err),
                                 _stream(stream)))


def moe_get_error(desc, ws, stream=None) -> int:
    """Synchronous convenience: enqueue the copy, synchronise the stream, return the code."""
    import torch
    code = ctypes.c_int32(-1)
    _check(load().moe_get_error(ctypes.byref(desc), _ptr(ws), ctypes.byref(code),
                                _stream(stream)))
    torch.cuda.synchronize()
    return code.value


def moe_clear_error(desc, ws, stream=None):
    _check(load().moe_clear_error(ctypes.byref(desc), _ptr(ws), _stream(stream)))


def moe_gemm_ctas(desc) -> int:
    return load().moe_gemm_ctas(ctypes.byref(desc))


def moe_launch_count() -> int:
    return int(load().moe_launch_count())


class Timeline:
    """Records a CUDA event after every library kernel launch (moe_timeline_begin/end) and
    turns consecutive event pairs into per-kernel durations."""

    def __init__(self, capacity: int):
        import torch
        self.capacity = capacity
        self.events = [torch.cuda.Event(enable_timing=True) for _ in range(capacity)]
        for e in self.events:           # torch creates events lazily: force creation
            e.record()
        torch.cuda.synchronize()
        self._handles = (_P * capacity)(*[e.cuda_event for e in self.events])
        self.ids = []

    def begin(self):
        _check(load().moe_timeline_begin(self._handles, self.capacity))

    def end(self) -> int:
        buf = (_I32 * self.capacity)()
        n = load().moe_timeline_end(buf)
        self.ids = list(buf[:n])
        return n

    def durations(self, start_event):
        """[(kernel_name, ms)] for each recorded launch, after a synchronize."""
        out = []
        prev = start_event
        for i, kid in enumerate(self.ids):
            out.append(((KERNEL_NAMES + MORE_KERNEL_NAMES)[kid], prev.elapsed_time(self.events[i])))
            prev = self.events[i]
        return out


# ------------------------------------------------------------------ buffer plumbing
def _made(index):
    """Ends a constructor that takes or fills memory of GPU `index` on its current stream: a first call on any
    other stream finds it filled, and done with what was there before. Within a capture both are the
    graph's."""
    import torch
    if not torch.cuda.is_current_stream_capturing():
        torch.cuda.current_stream(index).synchronize()


class MoELayer:
    """Owns the caller-side buffers of one layer (allocated with torch) and runs the C ABI
    calls on them. Weights: w1_packed [E, N1, H] bf16 (packed rows), w2 [E, F, H] bf16."""

    def __init__(self, desc: LayerDesc, device="cuda"):
        import torch
        load()
        self.desc = desc
        self.device = torch.device(device)
        self.layout = moe_workspace_layout(desc)
        self.ws_bytes = self.layout.total
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=self.device)
        d = desc
        self.N1 = d.F if d.activation == ACT["srelu"] else 2 * d.F
        T, E, k, H = d.T_max, d.E, d.k, d.H
        dev = self.device
        self.topk_ids = torch.empty(T, k, dtype=torch.int32, device=dev)
        self.topk_probs = torch.empty(T, k, dtype=torch.float32, device=dev)
        self.counts = torch.zeros(E, dtype=torch.int32, device=dev)
        self.y = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.dx = torch.empty(T, H, dtype=torch.bfloat16, device=dev)
        self.d_probs = torch.empty(T, k, dtype=torch.float32, device=dev)
        self.dw1 = None
        self.dw2 = None
        self.d_fc1_bias = None     # extras: [E, N1] fp32, logical order
        self.d_feat_scale = None   # extras: [E, F] fp32
        if self.ws.is_cuda:
            _made(self.ws.get_device())

    # views into the workspace -------------------------------------------------------
    def ws_view(self, name, dtype, shape):
        import torch
        off = getattr(self.layout, name)
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return self.ws[off:off + nbytes].view(dtype).view(*shape)

    def offsets(self):
        import torch
        return self.ws_view("offsets", torch.int32, (self.desc.E + 1,))

    # calls ---------------------------------------------------------------------------
    def route_permute(self, logits, x, T=None, stream=None):
        T = logits.shape[0] if T is None else T
        moe_route_permute(self.desc, T, logits, x, self.topk_ids, self.topk_probs, self.counts,
                          self.ws, self.ws_bytes, stream)

    def permute(self, topk_ids, topk_probs, x, T=None, stream=None):
        """In the place of route_permute, by a routing that is given (RouterTopK.forward's): experts
        int32 [T, k], ids outside [0, E) being dropped slots, and weights fp32 [T, k]. Writes
        self.counts; self.topk_ids and self.topk_probs stay route_permute's."""
        T = x.shape[0] if T is None else T
        if T > self.desc.T_max:
            raise ValueError(f"{T} tokens, but T_max is {self.desc.T_max}")
        index, k = self.ws.get_device(), self.desc.k
        _expect(topk_ids, "topk_ids", self.counts.dtype, (T, k), index)
        _expect(topk_probs, "topk_probs", self.topk_probs.dtype, (T, k), index)
        _expect(x, "x", self.y.dtype, (T, self.desc.H), index)
        moe_permute(self.desc, T, topk_ids, topk_probs, x, self.counts, self.ws, self.ws_bytes,
                    _call_stream(index, stream))

    def forward(self, w1_packed, w2, T, stream=None, fc1_bias=None, feat_scale=None):
        """fc1_bias fp32 [E, N1] (logical order) and feat_scale fp32 [E, F] for a layer made
        with the matching extras bits."""
        if self.desc.extras:
            moe_grouped_mlp_fwd_ex(self.desc, T, w1_packed, w2, fc1_bias, feat_scale, self.y,
                                   self.ws, self.ws_bytes, stream)
        else:
            moe_grouped_mlp_fwd(self.desc, T, w1_packed, w2, self.y, self.ws, self.ws_bytes,
                                stream)
        return self.y[:T]

    def backward(self, dy, w1_packed, w2, T, stream=None, feat_scale=None):
        import torch
        if self.dw1 is None:
            d = self.desc
            self.dw1 = torch.empty(d.E, self.N1, d.H, dtype=torch.bfloat16, device=self.device)
            self.dw2 = torch.empty(d.E, d.F, d.H, dtype=torch.bfloat16, device=self.device)
        if self.desc.extras:
            if self.d_fc1_bias is None:
                d = self.desc
                self.d_fc1_bias = (torch.empty(d.E, self.N1, dtype=torch.float32,
                                               device=self.device) if d.extras & 1 else None)
                self.d_feat_scale = (torch.empty(d.E, d.F, dtype=torch.float32,
                                                 device=self.device) if d.extras & 2 else None)
            moe_grouped_mlp_bwd_ex(self.desc, T, dy, w1_packed, w2, feat_scale, self.dx,
                                   self.dw1, self.dw2, self.d_probs, self.d_fc1_bias,
                                   self.d_feat_scale, self.ws, self.ws_bytes, stream)
        else:
            moe_grouped_mlp_bwd(self.desc, T, dy, w1_packed, w2, self.dx, self.dw1, self.dw2,
                                self.d_probs, self.ws, self.ws_bytes, stream)
        return self.dx[:T], self.dw1, self.dw2, self.d_probs[:T]

    def device_error(self, stream=None) -> int:
        return moe_get_error(self.desc, self.ws, stream)


def pack_w1(w1_logical, gated=True, ilv=64, stream=None):
    """w1_logical bf16 [E, H, N1] (torch, cuda) -> packed [E, N1, H] through the library."""
    import torch
    E, H, N1 = w1_logical.shape
    F = N1 // 2 if gated else N1
    out = torch.empty(E, N1, H, dtype=w1_logical.dtype, device=w1_logical.device)
    moe_pack_fc1_weight(w1_logical, out, E, H, F, gated, ilv, 0, stream)
    return out


# ------------------------------------------------------------------ operators around the layer
def _dtype_code(dtype) -> int:
    import torch
    code = {torch.bfloat16: 0, torch.float32: 1}.get(dtype)
    if code is None:
        raise ValueError(f"dtype must be bfloat16 or float32, not {dtype}")
    return code


def _gpu(device):
    """A GPU, with its index."""
    import torch
    dev = torch.device(device)
    if dev.type != "cuda":
        raise ValueError(f"device must be a GPU, not {dev}")
    return dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())


def _call_stream(index, stream):
    """The stream's handle, for a call whose memory is on GPU `index`: kernels go to the current
    one."""
    global _cuda
    if _cuda is None:
        import torch
        torch.cuda.current_device()  # initialises CUDA
        _cuda = torch._C
    if _cuda._cuda_getDevice() != index:
        raise ValueError(f"the buffers are on cuda:{index}, which is not the current device")
    return _cuda._cuda_getCurrentRawStream(index) if stream is None else _stream(stream)


def _torch_on(index, stream):
    """The context in which torch's own part of a call goes to the call's stream (None, torch's or a
    handle)."""
    import torch
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=index) if stream
                  else torch.cuda.default_stream(index))
    return torch.cuda.stream(stream)


def _expect(t, name, dtype, shape, index, rows=False):
    """A tensor argument's GPU, type, shape and strides: contiguous, or (rows) any row stride."""
    if t.get_device() != index:
        raise ValueError(f"{name}: must be on cuda:{index}, not {t.device}")
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, "
                         f"got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        if not rows or (t.shape[1] > 1 and t.stride(1) != 1) or (
                t.shape[0] > 1 and t.stride(0) < t.shape[1]):
            raise ValueError(f"{name}: strides {t.stride()} are not supported")
    return t


def _ld(t) -> int:
    """Row stride of a two-dimensional tensor (its width where it has a single row)."""
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _matrix(t, name, dtype, N, most, index):
    """Checks a matrix argument of N columns and up to `most` rows; its rows and row stride. One look at
    each of the tensor's attributes: a small call's time is the host's."""
    shape = t.shape
    if len(shape) != 2 or shape[0] > most:
        raise ValueError(f"{name}: expected at most {most} rows of {N}")
    if (t.get_device() != index or t.dtype != dtype or shape[1] != N or not t.is_contiguous()):
        _expect(t, name, dtype, (shape[0], N), index, rows=True)
        return shape[0], _ld(t)
    return shape[0], N


def _first(buf, n):
    """The first n rows of a buffer (the buffer itself when that is all of them)."""
    return buf if buf.shape[0] == n else buf[:n]


class RouterLoss:
    """Load-balance loss of a top-k router over up to T_max tokens, and the gradient of the
    router's logits (moe_router_loss_fwd / _bwd). Owns the results' buffers: they hold the last
    call's values. The backward takes counts from the last forward."""

    def __init__(self, E, k, T_max, coef=0.01, device="cuda"):
        import torch
        dev = self.device = _gpu(device)
        self._gpu = dev.index
        self.E, self.k, self.T_max, self.coef = E, k, T_max, float(coef)
        self.ws_bytes = moe_router_loss_workspace(E)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self.loss = torch.zeros(1, dtype=torch.float32, device=dev)
        self.counts = torch.zeros(E, dtype=torch.int32, device=dev)
        self.mean_prob = torch.zeros(E, dtype=torch.float32, device=dev)
        self.n_valid = torch.zeros(1, dtype=torch.int32, device=dev)
        self.d_logits = torch.empty(T_max, E, dtype=torch.float32, device=dev)
        self.has_counts = False
        # the buffers' addresses, taken once: a small call's time is the host's
        self._lib = _load_calls()
        self._p = {n: getattr(self, n).data_ptr() for n in
                   ("ws", "loss", "counts", "mean_prob", "n_valid", "d_logits")}
        _made(self._gpu)

    def _tokens(self, logits, topk_ids, token_mask):
        T = logits.shape[0]
        if T > self.T_max:
            raise ValueError(f"{T} tokens, but T_max is {self.T_max}")
        _expect(logits, "logits", self.loss.dtype, (T, self.E), self._gpu, rows=True)
        _expect(topk_ids, "topk_ids", self.counts.dtype, (T, self.k), self._gpu)
        if token_mask is not None:
            import torch
            if token_mask.dtype not in (torch.bool, torch.uint8):
                raise ValueError("token_mask must be bool or uint8")
            _expect(token_mask, "token_mask", token_mask.dtype, (T,), self._gpu)
        return T

    def forward(self, logits, topk_ids, token_mask=None, stream=None):
        """logits fp32 [T, E], topk_ids int32 [T, k], token_mask bool [T] (False: left out).
        Returns (loss [1], counts int32 [E], mean_prob [E])."""
        T = self._tokens(logits, topk_ids, token_mask)
        p = self._p
        _check(self._lib.moe_router_loss_fwd(
            logits.data_ptr(), _ld(logits), topk_ids.data_ptr(), _ptr(token_mask), T, self.E,
            self.k, self.coef, p["loss"], p["counts"], p["mean_prob"], p["n_valid"], p["ws"],
            self.ws_bytes, _call_stream(self._gpu, stream)))
        self.has_counts = True
        return self.loss, self.counts, self.mean_prob

    def backward(self, logits, topk_ids, topk_probs=None, d_probs=None, token_mask=None,
                 d_loss=None, stream=None):
        """Of the last forward's tokens, all or some. topk_probs and d_probs fp32 [T, k] (the
        layer's routing probabilities and the gradient its backward gives them), d_loss fp32 [1]
        (None: 1). Returns d_logits [T, E]."""
        if not self.has_counts:
            raise ValueError("backward needs a forward's counts")
        T = self._tokens(logits, topk_ids, token_mask)
        for t, name in ((topk_probs, "topk_probs"), (d_probs, "d_probs")):
            if t is not None:
                _expect(t, name, self.loss.dtype, (T, self.k), self._gpu)
        if d_loss is not None:
            _expect(d_loss, "d_loss", self.loss.dtype, d_loss.shape, self._gpu)
            if d_loss.numel() != 1:
                raise ValueError("d_loss must hold one value")
        p = self._p
        _check(self._lib.moe_router_loss_bwd(
            logits.data_ptr(), _ld(logits), topk_ids.data_ptr(), _ptr(topk_probs), _ptr(d_probs),
            _ptr(token_mask), T, self.E, self.k, self.coef, _ptr(d_loss), p["counts"],
            p["n_valid"], p["d_logits"], self.E, _call_stream(self._gpu, stream)))
        return _first(self.d_logits, T)


class RouterTopK:
    """The choice of experts for up to T_max tokens, and the gradient of its weights
    (moe_router_topk_fwd / _bwd). score "softmax" or "sigmoid"; groups: the topk_group best of n_group
    groups stay, each counting its best (group_top 1) or its two best experts (2); renorm: the chosen
    scores are divided by their sum. Owns the results' buffers: they hold the last call's values."""

    def __init__(self, E, k, T_max, score="sigmoid", n_group=1, topk_group=1, group_top=1,
                 renorm=True, scale=1.0, dtype=None, device="cuda"):
        import torch
        dev = self.device = _gpu(device)
        self._gpu = dev.index
        if score not in SCORE:
            raise ValueError(f"score must be one of {tuple(SCORE)}, not {score!r}")
        self.E, self.k, self.T_max = E, k, T_max
        self.dtype = torch.float32 if dtype is None else dtype
        self._code = _dtype_code(self.dtype)
        self.score, self.renorm, self.scale = score, bool(renorm), float(scale)
        self._score = SCORE[score]
        self._groups = n_group, topk_group, group_top
        self.topk_ids = torch.empty(T_max, k, dtype=torch.int32, device=dev)
        self.topk_weights = torch.empty(T_max, k, dtype=torch.float32, device=dev)
        self.counts = torch.zeros(E, dtype=torch.int32, device=dev)
        self.d_logits = None
        self.T = None  # tokens of the last forward
        self._lib = _load_calls()
        self._out = (self.topk_ids.data_ptr(), self.topk_weights.data_ptr(),
                     self.counts.data_ptr())
        _made(self._gpu)

    def forward(self, logits, bias=None, token_mask=None, stream=None):
        """logits [T, E], bias fp32 [E] (for the choice alone), token_mask bool [T] (False: ids -1,
        weights 0). Returns (topk_ids int32 [T, k], topk_weights fp32 [T, k], counts int32 [E])."""
        T, ld = _matrix(logits, "logits", self.dtype, self.E, self.T_max, self._gpu)
        if bias is not None:
            _expect(bias, "bias", self.topk_weights.dtype, (self.E,), self._gpu)
        if token_mask is not None:
            import torch
            if token_mask.dtype not in (torch.bool, torch.uint8):
                raise ValueError("token_mask must be bool or uint8")
            _expect(token_mask, "token_mask", token_mask.dtype, (T,), self._gpu)
        _check(self._lib.moe_router_topk_fwd(
            logits.data_ptr(), ld, self._code, None if bias is None else bias.data_ptr(),
            _ptr(token_mask), T, self.E, self.k, self._score, *self._groups, self.renorm, self.scale,
            *self._out, _call_stream(self._gpu, stream)))
        self.T = T
        if T == self.T_max:
            return self.topk_ids, self.topk_weights, self.counts
        return self.topk_ids[:T], self.topk_weights[:T], self.counts

    def backward(self, logits, d_weights, topk_ids=None, add_to=None, stream=None):
        """d_weights fp32 [T, k]; topk_ids: the forward's (None: those of the last forward, which had
        as many tokens or more); add_to fp32 [T, E] is added to the result (RouterLoss.backward's,
        say). Returns d_logits fp32 [T, E]."""
        T, ld = _matrix(logits, "logits", self.dtype, self.E, self.T_max, self._gpu)
        _expect(d_weights, "d_weights", self.topk_weights.dtype, (T, self.k), self._gpu)
        if topk_ids is None:
            if self.T is None or T > self.T:
                raise ValueError(f"no forward of {T} tokens has left topk_ids")
            topk_ids = self.topk_ids
        else:
            _expect(topk_ids, "topk_ids", self.topk_ids.dtype, (T, self.k), self._gpu)
        add = None, 0
        if add_to is not None:
            _expect(add_to, "add_to", d_weights.dtype, (T, self.E), self._gpu, rows=True)
            add = add_to.data_ptr(), _ld(add_to)
        if self.d_logits is None:
            import torch
            # what the current stream has given back may still be in use there
            with _torch_on(self._gpu, stream):
                self.d_logits = torch.empty(self.T_max, self.E, dtype=torch.float32,
                                            device=self.device)
        _check(self._lib.moe_router_topk_bwd(
            logits.data_ptr(), ld, self._code, topk_ids.data_ptr(), d_weights.data_ptr(), T, self.E,
            self.k, self._score, self.renorm, self.scale, *add, self.d_logits.data_ptr(), self.E,
            _call_stream(self._gpu, stream)))
        return self.d_logits if T == self.T_max else self.d_logits[:T]


class LayerNorm:
    """Layer norm over N features of up to M_max rows (moe_layernorm_fwd / _bwd). Owns the
    results' buffers: they hold the last call's values."""

    def __init__(self, N, M_max, dtype=None, weight_dtype=None, eps=1e-5, device="cuda"):
        import torch
        dev = self.device = _gpu(device)
        self._gpu = dev.index
        self.dtype = torch.bfloat16 if dtype is None else dtype
        self.weight_dtype = self.dtype if weight_dtype is None else weight_dtype
        self._codes = _dtype_code(self.dtype), _dtype_code(self.weight_dtype)
        self.N, self.M_max, self.eps = N, M_max, float(eps)
        self.y = torch.empty(M_max, N, dtype=self.dtype, device=dev)
        self.mean = torch.empty(M_max, dtype=torch.float32, device=dev)
        self.rstd = torch.empty(M_max, dtype=torch.float32, device=dev)
        self.dx = None
        self.M = None  # rows of the last forward
        self._lib = _load_calls()
        self._out = self.y.data_ptr(), N, self.mean.data_ptr(), self.rstd.data_ptr()
        _made(self._gpu)

    def _rows(self, x, name):
        if x.dim() != 2 or x.shape[0] > self.M_max:
            raise ValueError(f"{name}: expected at most {self.M_max} rows of {self.N}")
        return _expect(x, name, self.dtype, (x.shape[0], self.N), self._gpu, rows=True).shape[0]

    def _weight(self, w, name):
        if w is None:
            return None
        return _expect(w, name, self.weight_dtype, (self.N,), self._gpu)

    def forward(self, x, gamma=None, beta=None, stream=None):
        """Returns (y [M, N], mean [M], rstd [M])."""
        M = self._rows(x, "x")
        _check(self._lib.moe_layernorm_fwd(
            x.data_ptr(), _ld(x), _ptr(self._weight(gamma, "gamma")),
            _ptr(self._weight(beta, "beta")), *self._out, M, self.N, self.eps, *self._codes,
            _call_stream(self._gpu, stream)))
        self.M = M
        return _first(self.y, M), _first(self.mean, M), _first(self.rstd, M)

    def backward(self, dy, x, gamma=None, mean=None, rstd=None, stream=None):
        """mean, rstd: the forward's (None: those of the last forward, which had as many rows or
        more). Returns (dx [M, N], dgamma [N], dbeta [N])."""
        import torch
        M = self._rows(x, "x")
        if self._rows(dy, "dy") != M:
            raise ValueError("dy and x differ in rows")
        if (mean is None or rstd is None) and (self.M is None or M > self.M):
            raise ValueError(f"no forward of {M} rows has left mean and rstd")
        if mean is None:
            mean = self.mean
        else:
            _expect(mean, "mean", torch.float32, (M,), self._gpu)
        if rstd is None:
            rstd = self.rstd
        else:
            _expect(rstd, "rstd", torch.float32, (M,), self._gpu)
        if self.dx is None:
            self.ws_bytes = moe_layernorm_workspace(self.M_max, self.N)
            # what the current stream has given back may still be in use there
            with _torch_on(self._gpu, stream):
                self.dgamma = torch.empty(self.N, dtype=self.weight_dtype, device=self.device)
                self.dbeta = torch.empty(self.N, dtype=self.weight_dtype, device=self.device)
                self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=self.device)
                self.dx = torch.empty(self.M_max, self.N, dtype=self.dtype, device=self.device)
        _check(self._lib.moe_layernorm_bwd(
            dy.data_ptr(), _ld(dy), x.data_ptr(), _ld(x), _ptr(self._weight(gamma, "gamma")),
            mean.data_ptr(), rstd.data_ptr(), self.dx.data_ptr(), self.N, self.dgamma.data_ptr(),
            self.dbeta.data_ptr(), M, self.N, *self._codes, self.ws.data_ptr(), self.ws_bytes,
            _call_stream(self._gpu, stream)))
        return _first(self.dx, M), self.dgamma, self.dbeta


class ResidualNorm:
    """The residual stream around a block, x_new = x + scale * gate * (post_weight * N(o)) and
    h = weight * N(x_new) with root-mean-square norms N, over N features of up to M_max rows
    (moe_residual_norm_fwd / _bwd). dtype: the stream's (x), branch_dtype: o's and h's; post_norm: the
    branch is normed before it joins. Owns the results' buffers: they hold the last call's values."""

    def __init__(self, N, M_max, dtype=None, branch_dtype=None, weight_dtype=None,
                 post_norm=False, scale=1.0, eps=1e-6, device="cuda"):
        import torch
        dev = self.device = _gpu(device)
        self._gpu = dev.index
        self.dtype = torch.bfloat16 if dtype is None else dtype
        self.branch_dtype = self.dtype if branch_dtype is None else branch_dtype
        self.weight_dtype = self.branch_dtype if weight_dtype is None else weight_dtype
        self._codes = tuple(_dtype_code(t) for t in
                            (self.dtype, self.branch_dtype, self.weight_dtype))
        self.N, self.M_max = N, M_max
        self.post_norm, self.scale, self.eps = bool(post_norm), float(scale), float(eps)
        self._post = int(self.post_norm)
        self.x_new = None
        self.h = torch.empty(M_max, N, dtype=self.branch_dtype, device=dev)
        self.rstd = torch.empty(M_max, dtype=torch.float32, device=dev)
        self.rstd_post = torch.empty(M_max, dtype=torch.float32, device=dev)
        self.dx = None
        # rows whose rstd and rstd_post the last forward left
        self.M = self.M_post = None
        self._lib = _load_calls()
        self._out = self.h.data_ptr(), self.rstd_post.data_ptr(), self.rstd.data_ptr()
        _made(self._gpu)

    def _rows(self, x, name, dtype, M=None):
        """A matrix argument's rows, address and row stride."""
        rows, ld = _matrix(x, name, dtype, self.N, self.M_max, self._gpu)
        if M is not None and rows != M:
            raise ValueError(f"{name}: expected {M} rows, got {rows}")
        return rows, x.data_ptr(), ld

    def _weight(self, w, name):
        if w is None:
            return None
        return _expect(w, name, self.weight_dtype, (self.N,), self._gpu)

    def _branch(self, o, post_weight, gate, M):
        """Checks what belongs to a branch; its post norm (0 or 1), address and row stride."""
        if o is None:
            if post_weight is not None or gate is not None:
                raise ValueError("post_weight and gate need a branch o")
            return 0, None, 0
        _, at, ld = self._rows(o, "o", self.branch_dtype, M)
        if post_weight is not None:
            self._weight(post_weight, "post_weight")
        if gate is not None:
            _expect(gate, "gate", self.rstd.dtype, (M,), self._gpu)
        return self._post, at, ld

    def forward(self, x, o=None, weight=None, post_weight=None, gate=None, norm=True, stream=None):
        """x [M, N] of the stream, o [M, N] the branch that joins it (None: x_new is x), gate fp32
        [M]; norm=False: no h (the last block's sum). Returns (x_new [M, N], h [M, N] or None)."""
        M, at, ld = self._rows(x, "x", self.dtype)
        post, *branch = self._branch(o, post_weight, gate, M)
        if weight is not None:
            self._weight(weight, "weight")
        if not norm and (weight is not None or o is None):
            raise ValueError("without a norm there is a branch and no weight")
        h, rstd_post, rstd = self._out
        new = None
        if o is not None:
            if self.x_new is None:
                import torch
                # what the current stream has given back may still be in use there
                with _torch_on(self._gpu, stream):
                    self.x_new = torch.empty(self.M_max, self.N, dtype=self.dtype,
                                             device=self.device)
            new = self.x_new.data_ptr()
        _check(self._lib.moe_residual_norm_fwd(
            at, ld, *branch, None if post_weight is None else post_weight.data_ptr(),
            None if gate is None else gate.data_ptr(),
            None if weight is None else weight.data_ptr(), new, self.N, h if norm else None, self.N,
            rstd_post, rstd, M, self.N, self.scale, post, self.eps, *self._codes,
            _call_stream(self._gpu, stream)))
        self.M, self.M_post = (M if norm else None), (M if post else None)
        if o is not None:
            x = self.x_new if M == self.M_max else self.x_new[:M]
        if not norm:
            return x, None
        return x, self.h if M == self.M_max else self.h[:M]

    def _stats(self, given, name, own, M, rows):
        if given is not None:
            import torch
            return _expect(given, name, torch.float32, (M,), self._gpu).data_ptr()
        if rows is None or M > rows:
            raise ValueError(f"no forward of {M} rows has left {name}")
        return own.data_ptr()

    def backward(self, dh, x_new=None, o=None, weight=None, post_weight=None, gate=None,
                 dx_new=None, rstd=None, rstd_post=None, stream=None):
        """dh [M, N] the gradient of h (None: forward(norm=False)), dx_new that of x_new through
        everything else (None: 0), x_new and o the forward's; rstd, rstd_post: the forward's (None:
        those of the last forward, which had as many rows or more). Returns (dx, do, d_weight,
        d_post_weight, d_gate), None for what had no part."""
        import torch
        if dh is None and dx_new is None:
            raise ValueError("neither dh nor dx_new")
        none = None, 0
        if dh is None:
            M, *dxn = self._rows(dx_new, "dx_new", self.dtype)
            grad = none
        else:
            M, *grad = self._rows(dh, "dh", self.branch_dtype)
            dxn = none if dx_new is None else self._rows(dx_new, "dx_new", self.dtype, M)[1:]
        post, *branch = self._branch(o, post_weight, gate, M)
        if dh is None:
            if weight is not None:
                raise ValueError("weight needs dh")
            new, r = none, None
        else:
            if x_new is None:
                raise ValueError("dh needs x_new")
            new = self._rows(x_new, "x_new", self.dtype, M)[1:]
            r = self._stats(rstd, "rstd", self.rstd, M, self.M)
        rp = self._stats(rstd_post, "rstd_post", self.rstd_post, M, self.M_post) if post else None
        self._weight(weight, "weight")
        if self.dx is None:
            self.ws_bytes = moe_residual_norm_workspace(self.M_max, self.N)
            with _torch_on(self._gpu, stream):
                def make(dtype, *shape):
                    return torch.empty(*shape, dtype=dtype, device=self.device)
                self.dx = make(self.dtype, self.M_max, self.N)
                self.do = make(self.branch_dtype, self.M_max, self.N)
                self.d_weight = make(self.weight_dtype, self.N)
                self.d_post_weight = make(self.weight_dtype, self.N)
                self.d_gate = make(torch.float32, self.M_max)
                self.ws = make(torch.uint8, self.ws_bytes)
        do = None if o is None else self.do
        dw = None if weight is None else self.d_weight
        dwp = None if post_weight is None else self.d_post_weight
        dg = None if gate is None else self.d_gate
        _check(self._lib.moe_residual_norm_bwd(
            *grad, *dxn, *new, *branch, _ptr(post_weight), _ptr(gate), _ptr(weight), rp, r,
            self.dx.data_ptr(), self.N, _ptr(do), self.N, _ptr(dwp), _ptr(dw), _ptr(dg), M, self.N,
            self.scale, post, *self._codes, self.ws.data_ptr(), self.ws_bytes,
            _call_stream(self._gpu, stream)))
        return (_first(self.dx, M), None if do is None else _first(do, M), dw, dwp,
                None if dg is None else _first(dg, M))


def _overlap(spans) -> bool:
    """True where a tensor that is written shares memory with another one. (first byte, end, written)
    of each tensor."""
    end = end_written = 0
    for lo, hi, written in sorted(s for s in spans if s[1] > s[0]):
        if lo < (end if written else end_written):
            return True
        end = max(end, hi)
        if written:
            end_written = max(end_written, hi)
    return False


def _collide(grads, outs) -> bool:
    """True where a tensor that is written shares memory with another one. (address, bytes) of each
    gradient and of its out, which may be the gradient itself."""
    return _overlap([(o[0], o[0] + o[1], True) for o in outs]
                    + [(g[0], g[0] + g[1], False) for g, o in zip(grads, outs) if o != g])


class GradClip:
    """Global norm of a fixed list of gradient tensors, and clipping in place or into `outs`
    (moe_grad_clip). Holds references to the tensors: their memory stays where it is. A tensor that
    clipping writes shares memory with no other one."""

    def __init__(self, grads, outs=None):
        import torch
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError("outs must have one tensor for each gradient")
        for g, o in zip(self.grads, self.outs):
            if not (g.is_cuda and o.is_cuda and g.is_contiguous() and o.is_contiguous()):
                raise ValueError("gradients and outs must be on the GPU and contiguous")
            if g.device != self.grads[0].device or o.device != g.device:
                raise ValueError("gradients and outs must be on one device")
            if g.dtype != o.dtype or g.shape != o.shape:
                raise ValueError("an out differs from its gradient in type or shape")
        n = self.n = len(self.grads)
        dev = self.device = self.grads[0].device if n else _gpu("cuda")
        self._gpu = dev.index
        self._in = (_P * n)(*[g.data_ptr() for g in self.grads])
        self._out = (_P * n)(*[o.data_ptr() for o in self.outs])
        self._numel = (_I64 * n)(*[g.numel() for g in self.grads])
        self._types = (_I32 * n)(*[_dtype_code(g.dtype) for g in self.grads])
        self._at = [ctypes.addressof(a) for a in (self._in, self._out, self._numel, self._types)]
        self._shared = _collide(*[[(t.data_ptr(), t.numel() * t.element_size()) for t in ts]
                                  for ts in (self.grads, self.outs)])
        self.norm = torch.zeros(1, dtype=torch.float32, device=dev)
        self.ws_bytes = moe_grad_clip_workspace()
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=dev)
        self._lib = _load_calls()
        self._work = self.norm.data_ptr(), self.ws.data_ptr(), self.ws_bytes
        _made(self._gpu)

    def clip(self, max_norm, stream=None):
        """Returns the norm [1] (on the device). max_norm = inf only takes the norm."""
        if self._shared and max_norm != math.inf:
            raise ValueError("a tensor to be written shares memory with another one")
        at = self._at
        _check(self._lib.moe_grad_clip(self.n, at[0], None if max_norm == math.inf else at[1],
                                       at[2], at[3], max_norm, *self._work,
                                       _call_stream(self._gpu, stream)))
        return self.norm


class AdamW:
    """AdamW over a fixed list of weights and their gradients (moe_adamw_step). Holds references to
    the tensors: their memory stays where it is. Weights are fp32, or bf16 with an fp32 master
    (masters: one for each weight, None for fp32 ones; None: made here from the weights). State m and
    v in 32 bits, or 8: codes of m and of sqrt(v) with a scale byte for each 256 (m_exp, v_exp; see
    moments()), rounded at random from `seed`. weight_decay: a number, or one for each weight. lr: a
    number, or an fp32 tensor [1] on the GPU, which is read at each step (a captured one follows it).
    steps (int64 [1] on the GPU): the steps done. To resume, copy a checkpoint's masters, m, v, m_exp,
    v_exp and steps into those tensors."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state_bits=32, masters=None, seed=0):
        import torch
        self.params, self.grads = list(params), list(grads)
        n = self.n = len(self.params)
        decay = ([weight_decay] * n if isinstance(weight_decay, (int, float))
                 else list(weight_decay))
        masters = [None] * n if masters is None else list(masters)
        if len(self.grads) != n or len(decay) != n or len(masters) != n:
            raise ValueError("params, grads, masters and weight_decay differ in length")
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, not {state_bits}")
        if not 0 <= seed < 1 << 64:
            raise ValueError("seed must be in [0, 2^64)")
        dev = self.device = self.params[0].device if n else _gpu("cuda")
        for p, g, w in zip(self.params, self.grads, masters):
            for t in (p, g) if w is None else (p, g, w):
                if not t.is_cuda or not t.is_contiguous() or t.device != dev:
                    raise ValueError("tensors must be contiguous, on one GPU")
                if t.shape != p.shape:
                    raise ValueError("a gradient or master differs from its weight in shape")
            _dtype_code(p.dtype)
            _dtype_code(g.dtype)
            if w is not None and (w.dtype != torch.float32 or p.dtype == torch.float32):
                raise ValueError("a master is fp32, of a bf16 weight")
        self._gpu = dev.index
        self.state_bits, self.betas, self.eps, self.seed = state_bits, betas, eps, seed
        self.lr = lr
        self.masters = [p.detach().float() if w is None and p.dtype != torch.float32 else w
                        for p, w in zip(self.params, masters)]

        def states(dtype, per=1):
            return [torch.zeros(-(-p.numel() // per), dtype=dtype, device=dev)
                    for p in self.params]

        if state_bits == 32:
            self.m, self.v = states(torch.float32), states(torch.float32)
            self.m_exp = self.v_exp = [None] * n
        else:
            self.m, self.v = states(torch.uint8), states(torch.uint8)
            self.m_exp, self.v_exp = states(torch.uint8, 256), states(torch.uint8, 256)
        self._counters = torch.zeros(2, dtype=torch.int64, device=dev)
        self.steps = self._counters[:1]
        self._counters_at, self._f32 = self._counters.data_ptr(), torch.float32
        self._list = (AdamWTensor * n)(*[
            AdamWTensor(p.data_ptr(), _ptr(w), g.data_ptr(), m.data_ptr(), v.data_ptr(), _ptr(me),
                        _ptr(ve), p.numel(), _dtype_code(p.dtype), _dtype_code(g.dtype), d, 0)
            for p, w, g, m, v, me, ve, d in zip(self.params, self.masters, self.grads, self.m,
                                                self.v, self.m_exp, self.v_exp, decay)])
        self._at = ctypes.addressof(self._list)

        written = [*self.params, *self.masters, *self.m, *self.v, *self.m_exp, *self.v_exp]
        if _overlap([(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), w)
                     for ts, w in ((written, True), (self.grads, False)) for t in ts
                     if t is not None]):
            raise ValueError("a weight shares memory with another tensor")
        self._moments = None
        self._lib = _load_calls()
        _made(self._gpu)

    def step(self, norm=None, max_norm=math.inf, lr=None, stream=None):
        """One step. norm: GradClip's (fp32 [1] on the GPU): the gradients are multiplied by
        min(1, max_norm / (norm + 1e-6)), and a norm that is not finite skips the step. lr: another
        learning rate than the optimiser's, for this step."""
        lr = self.lr if lr is None else lr
        lr_dev = None
        if not isinstance(lr, (int, float)):
            lr_dev, lr = _expect(lr, "lr", self._f32, lr.shape, self._gpu), 0.0
            if lr_dev.numel() != 1:
                raise ValueError("lr must hold one value")
        if norm is not None:
            _expect(norm, "norm", self._f32, norm.shape, self._gpu)
            if norm.numel() != 1:
                raise ValueError("norm must hold one value")
        elif max_norm != math.inf:
            raise ValueError("max_norm needs the gradients' norm")
        _check(self._lib.moe_adamw_step(
            self.n, self._at, self.state_bits, lr, _ptr(lr_dev), *self.betas, self.eps,
            _ptr(norm), max_norm, self.seed, self._counters_at,
            _call_stream(self._gpu, stream)))

    def moments(self, stream=None):
        """The values that 8-bit states stand for: lists of m and of sqrt(v), bf16, in buffers that
        hold the last call's values."""
        import torch
        if self.state_bits != 8:
            raise ValueError("states in 32 bits are m and v themselves")
        if self._moments is None:
            with _torch_on(self._gpu, stream):
                self._moments = tuple([torch.empty(p.numel(), dtype=torch.bfloat16,
                                                   device=self.device) for p in self.params]
                                      for _ in range(2))
            self._moments_at = tuple((_P * self.n)(*[t.data_ptr() for t in ts])
                                     for ts in self._moments)
        _check(self._lib.moe_adamw_moments(
            self.n, self._at, *[ctypes.addressof(a) for a in self._moments_at],
            _call_stream(self._gpu, stream)))
        return self._moments


def _up(n, m) -> int:
    return (n + m - 1) // m * m


class Fp8Linear:
    """Dense layer y = x w^T in E4M3 with a scale for each block of 128 (fp8_block_*): w [N, K]
    bf16, x [M, K] bf16 with M <= M_max. Keeps the quantised weight (set_weight) and, for
    training, the quantised transposes of the last forward's x. Owns the results' buffers."""

    def __init__(self, N, K, M_max, train=True, device="cuda"):
        import torch
        dev = self.device = _gpu(device)
        self._gpu = dev.index
        self.N, self.K, self.M_max, self.train = N, K, M_max, train
        self.nb, self.kb = -(-N // 128), -(-K // 128)
        self._kp, self._np, self._mp = _up(K, 16), _up(N, 16), _up(max(M_max, 1), 16)

        def codes(rows, cols):
            return torch.empty(max(rows, 1), cols, dtype=torch.uint8, device=dev)

        def scales(blocks, n):
            return torch.empty(max(blocks, 1), n, dtype=torch.float32, device=dev)

        mb = -(-M_max // 128)
        self.wq, self.w_scale = codes(N, self._kp), scales(self.nb, self.kb)
        self.xq, self.x_scale = codes(M_max, self._kp), scales(self.kb, self._mp)
        self.y = torch.empty(M_max, N, dtype=torch.bfloat16, device=dev)
        self.err = torch.zeros(1, dtype=torch.int32, device=dev)
        self.M = None
        self.has_weight = False
        if train:
            self.wqt, self.wt_scale = codes(K, self._np), scales(self.kb, self.nb)
            self.xqt, self.xt_scale = codes(K, self._mp), scales(mb, _up(K, 4))
            self.dyq, self.dy_scale = codes(M_max, self._np), scales(self.nb, self._mp)
            self.dyqt, self.dyt_scale = codes(N, self._mp), scales(mb, _up(N, 4))
            self.dx = torch.empty(M_max, K, dtype=torch.bfloat16, device=dev)
            self.dw = torch.empty(N, K, dtype=torch.bfloat16, device=dev)

        # operands as (address of the codes, row stride, address of the scales, row stride)
        def operand(q, s):
            return q.data_ptr(), q.shape[1], s.data_ptr(), s.shape[1]

        self._lib = _load_calls()
        self._w, self._x = operand(self.wq, self.w_scale), operand(self.xq, self.x_scale)
        self._none = None, 0, None, 0
        self._xt = self._none
        if train:
            self._wt = operand(self.wqt, self.wt_scale)
            self._xt = operand(self.xqt, self.xt_scale)
            self._dy = operand(self.dyq, self.dy_scale)
            self._dyt = operand(self.dyqt, self.dyt_scale)
        _made(self._gpu)

    def set_weight(self, w, stream=None):
        """Quantise w bf16 [N, K] (both orders for training); again whenever w has changed."""
        import torch
        _expect(w, "w", torch.bfloat16, (self.N, self.K), self._gpu, rows=True)
        qt, ldqt, st, _ = self._wt if self.train else self._none
        _check(self._lib.fp8_block_quantize_weight(w.data_ptr(), _ld(w), self.N, self.K,
                                                   *self._w[:3], qt, ldqt, st,
                                                   _call_stream(self._gpu, stream)))
        self.has_weight = True

    def _quantize(self, x, M, N, row, col, stream):
        _check(self._lib.fp8_block_quantize_rows(x.data_ptr(), _ld(x), M, N, *row, *col, stream))

    def _product(self, a, b, blocks, c, M, N, K, stream):
        _check(self._lib.fp8_block_gemm(*a, *b, blocks, c.data_ptr(), N, 0, M, N, K,
                                        self.err.data_ptr(), stream))

    def forward(self, x, stream=None):
        """x bf16 [M, K] -> y bf16 [M, N]."""
        if not self.has_weight:
            raise ValueError("set_weight comes before forward")
        M = x.shape[0]
        if M > self.M_max:
            raise ValueError(f"{M} rows, but M_max is {self.M_max}")
        _expect(x, "x", self.y.dtype, (M, self.K), self._gpu, rows=True)
        stream = _call_stream(self._gpu, stream)
        self._quantize(x, M, self.K, self._x, self._xt, stream)
        self._product(self._x, self._w, 1, self.y, M, self.N, self.K, stream)
        self.M = M
        return _first(self.y, M)

    def backward(self, dy, stream=None):
        """dy bf16 [M, N] of the last forward's rows -> (dx bf16 [M, K], dw bf16 [N, K])."""
        if not self.train or self.M is None:
            raise ValueError("backward needs a layer made with train=True and a forward")
        M = self.M
        _expect(dy, "dy", self.y.dtype, (M, self.N), self._gpu, rows=True)
        if M == 0:
            with _torch_on(self._gpu, stream):
                return self.dx[:0], self.dw.zero_()
        stream = _call_stream(self._gpu, stream)
        self._quantize(dy, M, self.N, self._dy, self._dyt, stream)
        self._product(self._dy, self._wt, 1, self.dx, M, self.K, self.N, stream)
        self._product(self._dyt, self._xt, 0, self.dw, self.N, self.K, M, stream)
        return _first(self.dx, M), self.dw
