/*
 * moegmm.h - C ABI of the GB300 (sm_103a) fused grouped expert MLP of a Mixture-of-Experts
 * layer: routing + permutation, fused FC1 -> GLU -> probability scale -> FC2 forward, the
 * matching backward (BF16, MXFP8 or NVFP4 GEMM operands), the standalone MXFP8 and NVFP4
 * quantisers, and the operators around the layer in a training or serving step: the choice of
 * experts and the router's balance loss, layer norm, the norms around a block fused with its
 * residual sum, gradient clipping, AdamW, and a dense FP8 product with block-128 scales.
 *
 * Sources (by page title and section):
 *   [NV-blog] NVIDIA technical blog "Boosting MoE Training Throughput with Advanced Fusion
 *             Kernels" (zh-cn 借助高级融合内核提高 MoE 训练吞吐量): the three fused kernel
 *             families (GroupGemm + quantise; GroupGemm + activation + quantise/transpose;
 *             GroupGemm + dActivation + quantise/transpose), the SwiGLU equation and GLU weight
 *             repacking (GLU-epilogue section, Figure 2), device-resident per-group token
 *             counts (host-sync section), fused MXFP8 quantisation, dynamic scheduling and the
 *             configurable SM margin (kernel-to-pretraining section).
 *   [TE-MoE]  "NVIDIA Transformer Engine 优化 MoE 生物基础模型训练" (Transformer Engine MoE
 *             article): GroupedLinear with per-expert token counts, the per-expert loop with
 *             index_add (Challenge 1), MXFP8 format (Challenge 2, Figure 3), ScaledSwiGLU and
 *             the fused GroupedLinear -> ScaledSwiGLU -> GroupedLinear op (Challenge 3, Fig. 4).
 *   NVFP4 is named by [NV-blog] ("fused MXFP8 and NVFP4 quantisation": the forward kernel
 *   emits BF16 output plus a per-tensor amax, the backward kernel the amax of the
 *   Hadamard-rotated transposed output) but not defined there; the published format is used:
 *   E2M1 values, one unsigned E4M3 scale per 16 values, one fp32 scale per tensor (below).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers unless a name says host. Layouts are row-major.
 *     bf16 is passed as void* (2-byte IEEE bfloat16), e4m3 and e8m0 as uint8_t.
 *   - The caller owns every buffer, including the workspace `ws` (size from
 *     moe_workspace_size). No entry point allocates device memory or synchronises the host;
 *     all work is enqueued on `stream` (NULL = legacy default stream), so whole layer steps can
 *     be captured in a CUDA graph. Token counts and offsets never leave the device.
 *   - Host-side argument checks run before any launch and return MOE_ERR_INVALID_ARG or
 *     MOE_ERR_UNSUPPORTED with nothing enqueued. A CUDA launch error returns MOE_ERR_CUDA.
 *     Conditions only the device can see (routing capacity overflow, a bounded wait that timed
 *     out inside a kernel) set a sticky error word in the workspace, read by moe_get_error.
 *     No kernel traps, asserts or spins without a bound.
 *   - moe_last_error_string() describes the most recent host-side failure of this thread.
 */
#ifndef MOEGMM_H_
#define MOEGMM_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* cudaStream_t without pulling in the CUDA headers (same underlying type). */
typedef struct CUstream_st *moe_stream_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned pointer, k > E, ... */
  MOE_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. H not a multiple of 64)   */
  MOE_ERR_WORKSPACE = 3,    /* ws_bytes smaller than moe_workspace_size                  */
  MOE_ERR_CUDA = 4,         /* a CUDA runtime call or launch failed                       */
  MOE_ERR_DEVICE = 5        /* moe_get_error found a device-side error code               */
} moe_status_t;

/* Device error word codes (sticky until moe_clear_error). */
#define MOE_DEVERR_NONE 0
#define MOE_DEVERR_CAPACITY 1   /* routed rows exceeded the static capacity R_cap        */
#define MOE_DEVERR_TIMEOUT 2    /* a bounded barrier wait in a GEMM kernel gave up       */
#define MOE_DEVERR_BAD_ID 3     /* an expert id outside [0, E)                            */

/* GEMM operand precision. BF16: bf16 operands. MXFP8: E4M3 with one E8M0 scale per 32 values
 * (see mxfp8_quantize). NVFP4: E2M1 with one E4M3 scale per 16 values and one fp32 scale per
 * tensor (see nvfp4_quantize); the weight-gradient operands are Hadamard-rotated along the
 * tokens first (desc.rht_mask). Outputs and the saved FC1 output are bf16 in every case. */
typedef enum { MOE_PREC_BF16 = 0, MOE_PREC_MXFP8 = 1, MOE_PREC_NVFP4 = 2 } moe_precision_t;

/* Activations of [NV-blog] (SwiGLU, GeGLU, sReLU, "with clamp and scale options"):
 *   SWIGLU          a = lin * g * sigmoid(beta*g)                  (SwiGLU equation, b=c=0)
 *   CLAMPED_SWIGLU  g' = min(g, gate_max), l' = clamp(lin, lin_lo, lin_hi),
 *                   a = (l' + lin_offset) * g' * sigmoid(beta*g')
 *   GEGLU           a = lin * g * Phi(g)                           (exact erf GELU)
 *   SRELU           a = max(z, 0)^2, non-gated: FC1 has F (not 2F) output columns
 * The gradient passes a clamp at equality (the clamp is active strictly beyond a limit). */
typedef enum {
  MOE_ACT_SWIGLU = 0,
  MOE_ACT_CLAMPED_SWIGLU = 1,
  MOE_ACT_GEGLU = 2,
  MOE_ACT_SRELU = 3
} moe_activation_t;

/* Static description of one layer. Capacities are fixed here so that every call has the
 * same launch shapes (graph-capturable); the per-call token count T must be <= T_max. */
typedef struct {
  int32_t E;          /* experts (1..256)                                                */
  int32_t k;          /* experts per token (1..min(E,8))                                 */
  int32_t H;          /* hidden size, multiple of 64                                     */
  int32_t F;          /* expert FFN width, multiple of 64                                */
  int32_t T_max;      /* token capacity                                                  */
  int32_t precision;  /* moe_precision_t                                                 */
  int32_t activation; /* moe_activation_t                                                */
  float beta;         /* Swish beta (1.0 SwiGLU, 1.702 clamped GPT-OSS form)             */
  float gate_max;     /* clamped SwiGLU: upper clamp of the gate                         */
  float lin_lo;       /* clamped SwiGLU: lower clamp of the linear half                  */
  float lin_hi;       /* clamped SwiGLU: upper clamp of the linear half                  */
  float lin_offset;   /* clamped SwiGLU: added to the clamped linear half                */
  int32_t sm_margin;  /* SMs left free for concurrent kernels ([NV-blog] cluster margin) */
  int32_t ilv;        /* gate/linear interleave block of the packed W1 (32, 64 or 128)   */
  int32_t align;      /* expert segment alignment in rows: 32, 64 or 128 (BF16); 128
                         (MXFP8, NVFP4: segments start on 128-row scale slabs)            */
  int32_t recompute;  /* 1: keep no FC1 output between forward and backward; the FC2-dgrad
                         kernel recomputes it ([NV-blog] "What's next": activation
                         recomputation). Any precision and activation; 0 otherwise      */
  int32_t extras;     /* epilogue extras ([NV-blog] GLU-epilogue section: bias-vector addition
                         and feature scaling): bit 0 FC1 bias, bit 1 per-feature scale of the
                         activation output; used through the _ex entry points. Any
                         precision with a gated activation, without recompute; 0 otherwise */
  uint32_t rht_mask;  /* NVFP4: signs of the 16-point random Hadamard rotation applied along
                         the tokens to the weight-gradient operands (bit j set: the j-th row
                         of each 16-row block is negated before H16 / 4); drawn once by the
                         caller. Ignored by the other precisions                             */
  int32_t reuse_weights; /* MXFP8 / NVFP4: 1 = the forward does not quantise W1 and W2 again
                         but uses the block-scaled weight copies (and, NVFP4, their per-tensor
                         amaxes) that an earlier forward on the same workspace made from the
                         same BF16 master weights - the micro-batches of one gradient
                         accumulation step share them ([TE-MoE] Challenge 2: BF16 master
                         weights quantised before the low-precision GEMMs). The caller
                         guarantees the weights did not change since. 0 = quantise (always
                         correct). Ignored by BF16 layers                                    */
  int32_t pdl;        /* 1: every kernel the call enqueues is launched with programmatic stream
                         serialization (programmatic dependent launch), so that a kernel's CTAs
                         are scheduled while the previous kernel's last CTAs finish and only its
                         data reads wait for that kernel; 0: ordinary stream order. Results
                         are the same either way                                              */
} moe_layer_desc_t;

/* Byte offsets (from ws) of the intermediates that live in the workspace, for inspection
 * and tests. Offsets that do not apply to the layer's precision are SIZE_MAX. R_cap =
 * T_max*k + E*(align-1) rows. All row-indexed buffers use the permuted row order:
 * expert ascending, token ascending within an expert, each expert's segment starting at a
 * multiple of `align`; padding rows are zero and have probability 0. */
typedef struct {
  size_t total;          /* == moe_workspace_size                                        */
  int64_t R_cap;         /* row capacity                                                 */
  size_t err;            /* int32 device error word                                      */
  size_t offsets;        /* int32 [E+1] padded segment starts; offsets[E] = rows in use  */
  size_t row_of;         /* int32 [T_max*k] row of (token t, slot j) at t*k+j            */
  size_t src_of;         /* int32 [R_cap] t*k+j of a row, -1 for padding                 */
  size_t row_prob;       /* fp32 [R_cap] routing probability of a row, 0 for padding     */
  size_t x_perm;         /* bf16 [R_cap, H] gathered tokens                              */
  size_t z;              /* bf16 [R_cap, N1] FC1 output saved for backward (packed cols);
                            SIZE_MAX when the layer recomputes it                        */
  size_t a_s;            /* bf16 [R_cap, F] p * act(z), the FC2 input                    */
  size_t y_perm;         /* bf16 [R_cap, H] FC2 output before combine (shared with dx_perm) */
  size_t dy_perm;        /* bf16 [R_cap, H] gathered upstream gradient                   */
  size_t dz;             /* bf16 [R_cap, N1] gradient of z (packed cols)                 */
  size_t dx_perm;        /* bf16 [R_cap, H] FC1 dgrad output before combine              */
  size_t dprob_part;     /* fp32 [R_cap, ceil(F/128)] per-column-tile partial d_prob     */
  size_t ext_part;       /* fp32 [R_cap/32, N1 + F] per-32-row column sums of dZ and of
                            p * dA_s * a (extras only; SIZE_MAX otherwise)                 */
  size_t mx_base;        /* start of the MXFP8 operand copies (MXFP8 layers only)        */
  size_t nv_amax;        /* NVFP4 only: fp32 [16] per-tensor amax of each NVFP4 copy, in the
                            order x, x^T (rotated), W1, W2, a_s, a_s^T (rotated), dY, dY^T
                            (rotated), dZ, dZ^T (rotated); SIZE_MAX otherwise               */
  size_t nv_base;        /* start of the NVFP4 operand copies (NVFP4 layers only)        */
} moe_ws_layout_t;

/* Workspace bytes for a layer (0 if the description is invalid). */
size_t moe_workspace_size(const moe_layer_desc_t *desc);
/* Fill *out with the workspace layout. */
moe_status_t moe_workspace_layout(const moe_layer_desc_t *desc, moe_ws_layout_t *out);

/* Route + permute ([TE-MoE] Figure 1 top-k router; [NV-blog] host-sync section: per-group
 * token counts stay in device memory).
 *   logits     fp32 [T, E]   router logits
 *   x          bf16 [T, H]   tokens
 *   topk_ids   int32 [T, k]  out: experts by descending logit, ties to the lower index
 *   topk_probs fp32 [T, k]   out: softmax over the k chosen logits
 *   counts     int32 [E]     out: tokens routed to each expert
 * Writes offsets, row_of, src_of, row_prob and x_perm (and, for MXFP8 layers, the MXFP8
 * row-wise and column-wise copies of x_perm; for NVFP4 layers the amax and rotated amax of
 * x_perm, taken during the gather, and its row-wise and rotated transposed NVFP4 copies) into
 * ws. T in [0, T_max]. */
moe_status_t moe_route_permute(const moe_layer_desc_t *desc, int32_t T, const float *logits,
                               const void *x, int32_t *topk_ids, float *topk_probs,
                               int32_t *counts, void *ws, size_t ws_bytes, moe_stream_t stream);

/* Permute by a routing that is given (as moe_router_topk_fwd leaves it) in the place of the top-k
 * that moe_route_permute takes itself; everything else is as there, and the same calls follow it.
 *   topk_ids   int32 [T, k]  experts; an id outside [0, E) is a dropped slot: it gets no row (-1 in
 *              row_of), adds nothing to y and has d_probs 0. A token may name an expert twice:
 *              each slot gets a row of its own
 *   topk_probs fp32 [T, k]   weights of the experts' outputs
 *   counts     int32 [E]     out: rows of each expert
 * Rows are in the order expert, token, slot. T in [0, T_max]. */
moe_status_t moe_permute(const moe_layer_desc_t *desc, int32_t T, const int32_t *topk_ids,
                         const float *topk_probs, const void *x, int32_t *counts, void *ws,
                         size_t ws_bytes, moe_stream_t stream);

/* The routing maps of the last moe_route_permute on ws, copied into caller buffers (device
 * memory; [NV-blog] host-sync section: the per-expert counts and offsets stay on the device):
 *   offsets  int32 [E+1]    padded segment starts; offsets[E] = rows in use
 *   row_of   int32 [T*k]    permuted row of (token t, slot j) at t*k+j (-1: dropped by moe_permute)
 *   src_of   int32 [R_cap]  t*k+j of a permuted row, -1 for a padding row
 *   row_prob fp32  [R_cap]  routing probability of a permuted row, 0 for a padding row
 * R_cap as in moe_workspace_layout; rows at or beyond offsets[E] carry no routing (their
 * src_of / row_prob entries are left from earlier calls). Any of the four may be NULL (not
 * copied); each one given
 * must be 4-byte aligned. T must be the T of that moe_route_permute call, in [0, T_max]. One
 * kernel on `stream`, no host synchronisation, graph-capturable. Returns MOE_ERR_INVALID_ARG
 * for a bad description, workspace, T or pointer. */
moe_status_t moe_route_export(const moe_layer_desc_t *desc, const void *ws, size_t ws_bytes,
                              int32_t T, int32_t *offsets, int32_t *row_of, int32_t *src_of,
                              float *row_prob, moe_stream_t stream);

/* Fused grouped MLP forward ([NV-blog] kernel families 1 and 2, Figure 1; [TE-MoE]
 * GroupedLinear -> ScaledSwiGLU -> GroupedLinear):
 *   Z = X_e W1_e (FC1, grouped over experts from the device offsets), a = act(Z),
 *   a_s = p * a, Y_e = a_s W2_e (FC2), y[t] = sum_j Y[row_of[t,j]].
 *   w1_packed bf16 [E, N1, H]  FC1 weight, N1 = 2F (gated) or F (sReLU), rows in the packed
 *                              order of moe_pack_fc1_weight (gate/linear blocks interleaved)
 *   w2        bf16 [E, F, H]   FC2 weight (logical [F, H] per expert)
 *   y         bf16 [T, H]      out
 * Requires a preceding moe_route_permute or moe_permute on the same ws. Saves z and a_s in ws for the
 * backward. MXFP8 layers also quantise both weights (both directions) into ws first. NVFP4
 * layers take the weights' amax and NVFP4 copies (both directions) first; their FC1 kernel
 * also writes the amax and the rotated amax of a_s into ws (nv_amax), from which a_s's NVFP4
 * copies are made for FC2 and for the FC2 weight gradient. */
moe_status_t moe_grouped_mlp_fwd(const moe_layer_desc_t *desc, int32_t T, const void *w1_packed,
                                 const void *w2, void *y, void *ws, size_t ws_bytes,
                                 moe_stream_t stream);

/* Fused grouped MLP backward ([NV-blog] kernel family 3: FC2 dgrad + dActivation +
 * quantise/transpose; unfused weight-gradient GEMMs, Figure 1):
 *   dA_s = dY W2^T;  d_prob = sum_f dA_s * a;  dA = p * dA_s;  dZ = dact(Z, dA);
 *   dW2_e = a_s^T dY_e;  dW1_e = X_e^T dZ_e;  dX = dZ W1^T;  dx[t] = sum_j dX[row_of[t,j]].
 *   dy         bf16 [T, H]       upstream gradient of y
 *   dx         bf16 [T, H]       out
 *   dw1_packed bf16 [E, N1, H]   out, same packed row order as w1_packed (an expert with no
 *                                tokens gets exact zeros)
 *   dw2        bf16 [E, F, H]    out
 *   d_probs    fp32 [T, k]       out, gradient of topk_probs
 * Requires the forward's ws contents. NVFP4 layers gather dY together with its amax and
 * rotated amax, and their FC2-dgrad kernel writes dZ with its amax and rotated amax; every
 * GEMM then reads NVFP4 copies, the weight-gradient operands rotated along the tokens. */
moe_status_t moe_grouped_mlp_bwd(const moe_layer_desc_t *desc, int32_t T, const void *dy,
                                 const void *w1_packed, const void *w2, void *dx,
                                 void *dw1_packed, void *dw2, float *d_probs, void *ws,
                                 size_t ws_bytes, moe_stream_t stream);

/* Forward and backward with the epilogue extras (desc->extras; [NV-blog] GLU-epilogue
 * section: bias-vector addition and feature scaling; the SwiGLU equation's b and c):
 *   Z = X_e W1_e + b1_e (the bias in logical [gate | linear] column order, saved with Z),
 *   a_s = p * s_e * act(Z)  (s the per-feature scale of the activation output);
 *   backward: dA = p * s * dA_s, d_prob = sum_f dA_s * s * a,
 *             d_fc1_bias_e = sum over the expert's rows of dZ,
 *             d_feat_scale_e = sum over the expert's rows of p * dA_s * a.
 *   fc1_bias     fp32 [E, N1] logical order (bit 0 of extras; NULL otherwise)
 *   feat_scale   fp32 [E, F]  (bit 1; NULL otherwise)
 *   d_fc1_bias   fp32 [E, N1] out (bit 0; NULL otherwise)
 *   d_feat_scale fp32 [E, F]  out (bit 1; NULL otherwise)
 * Other arguments as moe_grouped_mlp_fwd / moe_grouped_mlp_bwd, which return
 * MOE_ERR_UNSUPPORTED for a layer with extras. The backward needs no bias (Z includes it).
 * Layers with a gated activation (BF16, MXFP8, NVFP4); in MXFP8 the scaled activation is
 * what the FC1 epilogue quantises, in NVFP4 what it emits in BF16 (with its amaxes), and the
 * dGLU epilogue takes the two column sums from the fp32 values, before dZ is rounded. */
moe_status_t moe_grouped_mlp_fwd_ex(const moe_layer_desc_t *desc, int32_t T,
                                    const void *w1_packed, const void *w2,
                                    const float *fc1_bias, const float *feat_scale, void *y,
                                    void *ws, size_t ws_bytes, moe_stream_t stream);
moe_status_t moe_grouped_mlp_bwd_ex(const moe_layer_desc_t *desc, int32_t T, const void *dy,
                                    const void *w1_packed, const void *w2,
                                    const float *feat_scale, void *dx, void *dw1_packed,
                                    void *dw2, float *d_probs, float *d_fc1_bias,
                                    float *d_feat_scale, void *ws, size_t ws_bytes,
                                    moe_stream_t stream);

/* Route + permute without any device allocation and without a workspace. The pages have no
 * counterpart of this entry point; it exists for callers that cannot call cudaMalloc, such as
 * plugins hosted by a framework that owns the whole device memory pool and forbids
 * allocations of its own, or code that runs where an allocation would stall or is not
 * allowed (for example while a CUDA graph is being recorded).
 * It computes the same results as moe_route_permute (topk_ids, topk_probs, counts, and the
 * gathered tokens) but writes the padded offsets and the gathered tokens to caller buffers:
 *   offsets  int32 [E+1]                  out: padded expert segment starts
 *   x_perm   bf16  [x_perm_rows, H]       out: x_perm_rows >= T_max*k + E*(align-1); same
 *                                          rows as moe_route_permute's workspace x_perm
 * Its scratch (row map, per-row source and probability, an error word) is a fixed
 * file-scope device array of about 1.6 MB inside the library, held by every GPU that loads
 * the library until the process exits. Limit: T_max*k <= 131072 routed (token, expert)
 * pairs, which with E <= 256 and any segment alignment (32, 64, 128) keeps R_cap within the
 * array's 163584 rows; larger descriptions return MOE_ERR_UNSUPPORTED before any launch. Only
 * BF16 layers. The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current, and looks it up again when the device's
 * context has changed since (after cudaDeviceReset, for example); make the first call after
 * such a change before any stream capture. All calls on a device share the array and it keeps
 * the last call's contents: the
 * error word and counts are cleared at the start of every call, and calls whose execution
 * overlaps on the GPU (for example on two streams) race. Capacity errors detected on the
 * device are not reported by this entry point (they cannot occur when T <= T_max). */
moe_status_t moe_route_permute_noalloc(const moe_layer_desc_t *desc, int32_t T,
                                       const float *logits, const void *x, int32_t *topk_ids,
                                       float *topk_probs, int32_t *counts, int32_t *offsets,
                                       void *x_perm, int64_t x_perm_rows, moe_stream_t stream);

/* Standalone MXFP8 quantiser ([TE-MoE] Challenge 2, Figure 3: E4M3 elements with one E8M0
 * scale per 32 contiguous values):
 *   scale exponent e = clamp(floor(log2(amax)) - 8, -127, 127) (e = -127 when amax = 0),
 *   scale byte e + 127, q = E4M3(v / 2^e) rounded to nearest even, saturating at +-448.
 *   in      bf16 [M, N]
 *   rowwise:  q_row  e4m3 [M, N]       blocks of 32 along N; s_row e8m0 [M, N/32]
 *   colwise:  q_col  e4m3 [M, N]       blocks of 32 along M (same layout as in);
 *             s_col  e8m0 [N, M/32]    without groups: blocks start at every 32nd row
 *   group_offsets  int32 [num_groups + 1], DEVICE memory, or NULL: rows [off[g], off[g+1])
 *             form group g (off[0] = 0, non-decreasing, off[num_groups] = M; the per-expert
 *             token counts of a GroupedLinear, [TE-MoE] Challenge 1, need not be multiples
 *             of 32). Column-wise blocks then restart at each group's first row: block i of
 *             group g is rows off[g] + 32i .. min(off[g] + 32i + 32, off[g+1]) (a short last
 *             block is quantised as if padded with zeros), and
 *             s_col e8m0 [N, nb], nb = 4 * ceil((ceil(M/32) + num_groups) / 4): the scale of
 *             column c, block (g, i) is s_col[c * nb + off[g]/32 + g + i] (integer division);
 *             entries no block owns are written 0. The offsets are read on the device only
 *             (no host sync); offsets outside [0, M] are clamped, and offsets that break the
 *             rules above give unspecified (but in-bounds) results. The row-wise copy does not
 *             depend on the groups. num_groups must be in [1, 65536] when group_offsets is set.
 * N must be a multiple of 32; M a multiple of 32 for colwise without groups (any M with
 * groups); in and q_col 16-byte aligned and s_col 4-byte aligned with groups; the pointers of
 * an unused direction may be NULL. Bit-exact: the result does not depend on the launch. */
moe_status_t mxfp8_quantize(const void *in, int64_t M, int64_t N, int32_t rowwise,
                            int32_t colwise, const int32_t *group_offsets, int32_t num_groups,
                            uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                            moe_stream_t stream);

/* NVFP4 per-tensor amax ([NV-blog] "fused MXFP8 and NVFP4 quantisation": the scale of an NVFP4
 * tensor needs its amax first).
 *   in        bf16 [M, N]
 *   amax      fp32 [1] out: max |in|
 *   amax_rht  fp32 [1] out (may be NULL): max |y| over y = (1/4) H16 diag(d) x for every
 *             column and every block of 16 consecutive rows (x the block's 16 values, H16
 *             the Sylvester Hadamard matrix, d_j = -1 where bit j of sign_mask is set)
 * Both outputs are overwritten (the call zeroes them first). N must be a multiple of 64 (and
 * below 64 * 65536); M a multiple of 16 when amax_rht is given. M = 0 gives 0. */
moe_status_t nvfp4_amax(const void *in, int64_t M, int64_t N, uint32_t sign_mask, float *amax,
                        float *amax_rht, moe_stream_t stream);

/* Standalone NVFP4 quantiser. Per tensor S = min(2688 / amax, FLT_MAX) (2688 = 6 * 448); per
 * block of 16 values s_b = E4M3(fp32(amax_b / 6) * S) (round to nearest even, saturating);
 * per value q = E2M1(v * fp32(S / s_b)) (nearest even, saturating at +-6; factor 0 when
 * s_b = 0). Each step is one IEEE fp32 operation. The value represented is E2M1(q) * s_b / S.
 *   in        bf16 [M, N]
 *   amax_row  fp32 [1] device: the amax S is computed from for the row-wise copy
 *   amax_col  fp32 [1] device: the same for the transposed copy (the rotated amax when rht)
 *   row-wise:    q_row  [M, N/2] bytes, two E2M1 codes a byte (even index in the low nibble),
 *                       blocks of 16 along N;
 *                s_row  E4M3 scales in the MMA slab layout: the scale of (row r, block j) at
 *                       byte ((j/4) * M + perm(r)) * 4 + j%4, perm(r) = (r & ~127) |
 *                       ((r & 31) << 2) | ((r >> 5) & 3); (N/64) * M * 4 bytes
 *   transposed:  q_col  [N, M/2] bytes: row n holds column n of in, blocks of 16 along M,
 *                       each block first rotated as in nvfp4_amax when rht != 0;
 *                s_col  slab layout of (row n, block j): (M/64) * round128(N) * 4 bytes
 * M must be a positive multiple of 128 and N of 64; q_row and q_col 32-byte aligned, s_row
 * and s_col 4-byte aligned. q_row/s_row or q_col/s_col may both be NULL to skip that copy (its
 * amax pointer may then be NULL). Bit-exact: the result does not depend on the launch. */
moe_status_t nvfp4_quantize(const void *in, int64_t M, int64_t N, const float *amax_row,
                            const float *amax_col, int32_t rht, uint32_t sign_mask,
                            uint8_t *q_row, uint8_t *s_row, uint8_t *q_col, uint8_t *s_col,
                            moe_stream_t stream);

/* GLU weight repacking ([NV-blog] GLU-epilogue section and Figure 2: the gate and linear
 * columns are repacked so one output tile holds half a tile of each; done once, before
 * training or at checkpoint load).
 *   forward (inverse = 0): w1_logical bf16 [E, H, N1] -> w1_packed bf16 [E, N1, H]
 *   inverse (inverse = 1): w1_packed -> w1_logical
 * Gated (N1 = 2F): packed row p belongs to block b = p / ilv; even blocks are gate columns
 * (b/2)*ilv + p%ilv, odd blocks the linear columns F + (b/2)*ilv + p%ilv. sReLU (N1 = F):
 * packed = transpose. ilv must be a multiple of 32 that divides F. */
moe_status_t moe_pack_fc1_weight(const void *w1_src, void *w1_dst, int32_t E, int32_t H,
                                 int32_t F, int32_t gated, int32_t ilv, int32_t inverse,
                                 moe_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * Operators around the expert layer: the choice of experts and the router's balance loss, layer
 * norm and residual norm, gradient clipping, AdamW, and a dense product in 8-bit floating point
 * with a scale for each block of 128. They take no
 * layer description; the conventions at the top of this file hold (caller-owned device memory,
 * no synchronisation, graph-capturable, checks before any launch). Results do not depend on the
 * timing of the launch: sums are taken in a fixed order.
 * ------------------------------------------------------------------------------------------ */
typedef enum { MOE_DT_BF16 = 0, MOE_DT_FP32 = 1 } moe_dtype_t;

/* Choice of experts. With l the E logits of a token (NaN is read as -inf):
 *   score s_e   MOE_SCORE_SIGMOID: 1 / (1 + exp(-l_e)).  MOE_SCORE_SOFTMAX: exp(l_e - max l), 1
 *               where l_e is the maximum, times the reciprocal of their sum; the sum takes
 *               neighbours in pairs, then pairs of pairs, zeros filling up to a power of two
 *   value v_e   s_e + bias[e] (NaN is read as -inf), or s_e without a bias
 *   choice c_e  v_e, or without a bias l_e itself, which has the scores' order
 *   groups      the experts in n_group groups of E / n_group neighbours; a group counts the largest
 *               c of its experts (group_top 1) or the sum of its two largest v (group_top 2; NaN is
 *               read as -inf); the topk_group largest groups stay (ties to the lower one)
 *   topk_ids    the k experts of those groups by descending c (ties to the lower index)
 *   weights     scale * s_j;  with renorm, sigmoid: scale * s_j / (sum of the chosen s + 1e-20),
 *               softmax: scale * softmax over the chosen logits (those equal to their maximum
 *               weigh 1 before normalisation)
 * Each step up to the choice is one rounded fp32 operation (exp: CUDA's expf), so that the choice
 * between near values does not depend on the launch. A token whose mask is 0 gets ids -1 (dropped
 * slots to every function here) and weights 0, and is not counted.
 *   logits       [T, E] of logits_dtype (moe_dtype_t), row stride ld_logits >= E
 *   bias         fp32 [E] or NULL: it takes part in the choice alone
 *   token_mask   uint8 [T] or NULL: all tokens
 *   topk_ids     int32 [T, k] out;  topk_weights fp32 [T, k] out
 *   counts       int32 [E] out, or NULL: (token, slot) pairs of each expert
 * E in [1, 256], k in [1, min(E, 8)], n_group a divisor of E, topk_group in [1, n_group] with
 * topk_group * E / n_group >= k, group_top 1 or 2 (2: at least two experts a group); T >= 0. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_t;
moe_status_t moe_router_topk_fwd(const void *logits, int64_t ld_logits, int32_t logits_dtype,
                                 const float *bias, const uint8_t *token_mask, int32_t T,
                                 int32_t E, int32_t k, int32_t score, int32_t n_group,
                                 int32_t topk_group, int32_t group_top, int32_t renorm,
                                 float scale, int32_t *topk_ids, float *topk_weights,
                                 int32_t *counts, moe_stream_t stream);
/* Gradient of the logits through the weights (the choice is constant), u_j = scale * d_weights_j:
 *   sigmoid:          ds_j = u_j, d_e = ds_j s_j (1 - s_j) at the chosen experts;
 *   sigmoid, renorm:  ds_j = (u_j - sum_i u_i s_i / S) / S,  S = sum of the chosen s + 1e-20
 *   softmax:          d_e = p_e (u_e - sum_j u_j p_j), u_e = 0 for experts that are not chosen
 *   softmax, renorm:  d_e = w_j (u_j - sum_i w_i u_i) at the chosen experts, w their softmax
 * Dropped slots (ids outside [0, E)) take no part; slots that name the same expert add up.
 *   topk_ids    int32 [T, k], d_weights fp32 [T, k] (moe_grouped_mlp_bwd's d_probs)
 *   add_to      fp32 [T, E], row stride ld_add >= E, or NULL: added to the result (the balance
 *               loss's gradient from moe_router_loss_bwd, say); may be d_logits
 *   d_logits    fp32 [T, E] out, row stride ld_d >= E, written whole; it shares memory with no other rows
 *               of add_to or of the logits */
moe_status_t moe_router_topk_bwd(const void *logits, int64_t ld_logits, int32_t logits_dtype,
                                 const int32_t *topk_ids, const float *d_weights, int32_t T,
                                 int32_t E, int32_t k, int32_t score, int32_t renorm, float scale,
                                 const float *add_to, int64_t ld_add, float *d_logits,
                                 int64_t ld_d, moe_stream_t stream);

/* Load-balance loss of a top-k router and the counts it is made of. With p[t] the softmax of
 * token t's E logits, over the n tokens whose mask is set:
 *   counts[e]    = number of (token, slot) pairs with topk_ids == e
 *   mean_prob[e] = (1/n) sum_t p[t][e],     f[e] = E * counts[e] / (k * n)
 *   loss         = coef * sum_e f[e] * mean_prob[e]       (1 * coef for a uniform router)
 *   logits     fp32 [T, E], row stride ld_logits >= E. NaN is read as -inf; a logit equal to its
 *              row's maximum has weight 1 before normalisation (the softmax's limit for infinite
 *              maxima), as in moe_route_permute
 *   topk_ids   int32 [T, k]; an id outside [0, E) is a dropped slot and counts nowhere
 *   token_mask uint8 [T], 0 = left out (padding), or NULL: all tokens count
 *   loss fp32 [1], counts int32 [E], mean_prob fp32 [E], n_valid int32 [1]: outputs. Without a
 *              valid token all four are 0.
 * E in [1, 256], k in [1, min(E, 8)], T >= 0. ws: moe_router_loss_workspace(E) bytes, 16-byte
 * aligned, no initial value needed. */
size_t moe_router_loss_workspace(int32_t E);
moe_status_t moe_router_loss_fwd(const float *logits, int64_t ld_logits, const int32_t *topk_ids,
                                 const uint8_t *token_mask, int32_t T, int32_t E, int32_t k,
                                 float coef, float *loss, int32_t *counts, float *mean_prob,
                                 int32_t *n_valid, void *ws, size_t ws_bytes,
                                 moe_stream_t stream);
/* Gradient of the router's logits: the loss's (f held constant, as it is piecewise constant)
 * and, with topk_probs and d_probs, that of the chosen probabilities w = softmax over the k
 * chosen logits (d_probs as moe_grouped_mlp_bwd returns it), g = *d_loss (NULL: 1):
 *   d_logits[t][e] = mask[t] * g * coef / n * p[t][e] * (f[e] - sum_i p[t][i] f[i])
 *                  + sum over slots j with topk_ids[t][j] == e of w[j] * (d[j] - sum_i w[i] d[i])
 *   topk_probs, d_probs fp32 [T, k], both or neither NULL (the mask does not apply to them)
 *   counts, n_valid     as written by moe_router_loss_fwd (device memory)
 *   d_logits            fp32 [T, E], row stride ld_d >= E, written whole */
moe_status_t moe_router_loss_bwd(const float *logits, int64_t ld_logits, const int32_t *topk_ids,
                                 const float *topk_probs, const float *d_probs,
                                 const uint8_t *token_mask, int32_t T, int32_t E, int32_t k,
                                 float coef, const float *d_loss, const int32_t *counts,
                                 const int32_t *n_valid, float *d_logits, int64_t ld_d,
                                 moe_stream_t stream);

/* Layer norm over the last dimension: mean and rstd = 1 / sqrt(var + eps) of each row (biased
 * variance about the mean), y = (x - mean) * rstd * gamma + beta.
 *   x, y         [M, N] of x_dtype, row strides ldx, ldy >= N; y may be x
 *   gamma, beta  [N] of w_dtype, each may be NULL (1, 0)
 *   mean, rstd   fp32 [M] out, each may be NULL (a backward pass needs both)
 * x_dtype BF16 with w_dtype BF16 or FP32, or both FP32. eps >= 0. M >= 0, N >= 1. */
moe_status_t moe_layernorm_fwd(const void *x, int64_t ldx, const void *gamma, const void *beta,
                               void *y, int64_t ldy, float *mean, float *rstd, int64_t M,
                               int64_t N, float eps, int32_t x_dtype, int32_t w_dtype,
                               moe_stream_t stream);
/* Its backward pass from the saved mean and rstd, with h = (x - mean) * rstd, u = dy * gamma:
 *   dx = rstd * (u - mean_n(u) - h * mean_n(u * h)),  dgamma = sum_m dy * h,  dbeta = sum_m dy
 *   dx            [M, N] of x_dtype, row stride lddx; may be dy or x
 *   dgamma, dbeta [N] of w_dtype out, each may be NULL; summed in fp32 in a fixed order
 *                 (zeros for M = 0)
 * ws: moe_layernorm_workspace(M, N) bytes, 16-byte aligned (may be NULL when both weight
 * gradients are). */
size_t moe_layernorm_workspace(int64_t M, int64_t N);
moe_status_t moe_layernorm_bwd(const void *dy, int64_t lddy, const void *x, int64_t ldx,
                               const void *gamma, const float *mean, const float *rstd, void *dx,
                               int64_t lddx, void *dgamma, void *dbeta, int64_t M, int64_t N,
                               int32_t x_dtype, int32_t w_dtype, void *ws, size_t ws_bytes,
                               moe_stream_t stream);

/* The residual stream around a block, with root-mean-square norms N(a) = a / sqrt(mean(a^2) + eps)
 * (over a row) after the block and before the next one:
 *   u     = post_weight * N(o) (post_norm 1), or post_weight * o (post_norm 0: a gate a feature)
 *   x_new = x + scale * gate[m] * u
 *   h     = weight * N(x_new), of x_new as it is stored
 *   x, x_new     [M, N] of x_dtype, row strides ldx, ldxn >= N; x_new may be x. Without a branch
 *                (o NULL) x_new is x: x_new must be NULL, and h alone is made
 *   o, h         [M, N] of o_dtype, row strides ldo, ldh >= N; o may be NULL (no branch), h may be
 *                NULL (no norm: the last block's sum); h may be o. What is written shares memory with
 *                nothing else, but for a tensor that it is in the place of, row for row
 *   post_weight, weight  [N] of w_dtype, each may be NULL (1)
 *   gate         fp32 [M] or NULL (1)
 *   rstd_post, rstd  fp32 [M] out, each may be NULL: 1 / sqrt(mean + eps) of the two norms (rstd_post
 *                is not written without a post norm), which a backward pass needs
 * x_dtype, o_dtype: both BF16, both FP32, or FP32 and BF16. w_dtype BF16 or FP32 with o_dtype BF16,
 * FP32 otherwise. eps >= 0, M >= 0, N >= 1. The sums of squares are fp32 ones. */
moe_status_t moe_residual_norm_fwd(const void *x, int64_t ldx, const void *o, int64_t ldo,
                                   const void *post_weight, const float *gate,
                                   const void *weight, void *x_new, int64_t ldxn, void *h,
                                   int64_t ldh, float *rstd_post, float *rstd, int64_t M,
                                   int64_t N, float scale, int32_t post_norm, float eps,
                                   int32_t x_dtype, int32_t o_dtype, int32_t w_dtype,
                                   moe_stream_t stream);
/* Its backward pass, from x_new and o as the forward left them, with y = x_new * rstd,
 * z = o * rstd_post (post_norm 0: o) and q = scale * gate:
 *   dx  = dx_new + rstd (dh weight - y mean_n(dh weight y))     (the gradient of x, and of x_new)
 *   do  = q rstd_post (e - z mean_n(e z)),  e = dx post_weight  (post_norm 0: q e)
 *   d_weight = sum_m dh y;  d_post_weight = sum_m q dx z;  d_gate[m] = scale sum_n e z
 *   dh, o, do    [M, N] of o_dtype, dx_new, x_new, dx of x_dtype, row strides >= N. dh NULL: no norm
 *                follows; dx_new NULL: nothing else reads x_new; not both. o NULL: no branch (do,
 *                d_post_weight, d_gate, post_weight, gate and rstd_post are NULL too). x_new and
 *                rstd may be NULL without dh
 *   dx may be dx_new, do may be dh or o, else what is written shares no memory with other tensors (as in
 *                the forward); dx NULL: not written (it is dx_new when there is no dh)
 *   d_weight, d_post_weight [N] of w_dtype out, each may be NULL; summed in fp32 in a fixed order
 *                (zeros for M = 0).  d_gate fp32 [M] out or NULL
 * ws: moe_residual_norm_workspace(M, N) bytes, 16-byte aligned (may be NULL when both weight
 * gradients are). */
size_t moe_residual_norm_workspace(int64_t M, int64_t N);
moe_status_t moe_residual_norm_bwd(const void *dh, int64_t lddh, const void *dx_new,
                                   int64_t lddxn, const void *x_new, int64_t ldxn, const void *o,
                                   int64_t ldo, const void *post_weight, const float *gate,
                                   const void *weight, const float *rstd_post, const float *rstd,
                                   void *dx, int64_t lddx, void *d_o, int64_t lddo,
                                   void *d_post_weight, void *d_weight, float *d_gate, int64_t M,
                                   int64_t N, float scale, int32_t post_norm, int32_t x_dtype,
                                   int32_t o_dtype, int32_t w_dtype, void *ws, size_t ws_bytes,
                                   moe_stream_t stream);

/* Global gradient norm over n tensors, and clipping:
 *   norm = sqrt(sum over all elements of g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c*g
 * A NaN anywhere makes norm and c NaN; an infinite element makes c 0 (and itself NaN). Finite
 * gradients of any magnitude have a finite sum: up to 32 squares at a time are added in fp32, those
 * sums as pairs of fp32 numbers, and what leaves fp32's range in fp64. norm is rounded to fp32:
 * above 3.4e38 it is returned as +inf, while c and out are those of the finite norm.
 *   grads   HOST array of n device pointers (element-aligned; a 16-byte aligned start is not
 *           needed), numel HOST array of their element counts (>= 0), dtypes HOST array of
 *           moe_dtype_t
 *   outs    HOST array of n device pointers of the same types, or NULL: in place. outs[i] may
 *           equal grads[i]; otherwise tensors must not overlap. In place, c = 1 writes nothing.
 *   max_norm > 0; +inf: the norm alone is taken and outs must be NULL
 *   norm    fp32 [1] device, out
 * The three arrays are read before the call returns. n in [0, 65536].
 * ws: moe_grad_clip_workspace() bytes, 16-byte aligned, no initial value needed. */
size_t moe_grad_clip_workspace(void);
moe_status_t moe_grad_clip(int32_t n, const void *const *grads, void *const *outs,
                           const int64_t *numel, const int32_t *dtypes, float max_norm,
                           float *norm, void *ws, size_t ws_bytes, moe_stream_t stream);

/* One AdamW step over n tensors. With t the steps done before plus 1, g the gradient times the clip
 * factor, p the fp32 value of a weight (its master where it has one):
 *   m <- beta1 m + (1 - beta1) g;  v <- beta2 v + ((1 - beta2) g) g
 *   p <- (p - lr decay p) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * each product, sum and root of m and v one rounded fp32 operation.
 * States in 8 bits hold m and r = sqrt(v) (v = r r when read). 256 values in a row share a scale byte
 * b; a code's magnitude c (1..127 for m, under a sign bit; 1..255 for r) stands for the fp32 number
 * whose bits are (c + 8 b + 7 - C) << 20, C = 127 or 255: eight values a power of two, 16 or 32 powers
 * of two down from 2^(b - 127) * 1.875; c = 0 is 0. b is the smallest that holds the block's largest
 * value rounded up (at least 32), 255 for a block with a NaN or an infinity, whose values are NaN.
 * Values are rounded to one of their two neighbours at random, in proportion to their distance
 * (sixteen random bits: the low half of a 32-bit word for m, the high half for r), so that small
 * changes are not lost. The word of element e of tensor i in step t is
 *   mix(low32(e) ^ mix(high32(e) ^ mix(i + mix(low32(t) ^ mix(low32(seed) ^ mix(high32(seed)))))))
 * with mix(x): x ^= x >> 16; x *= 0xf75341d5; x ^= x >> 15; x *= 0x99d5d0a1; x ^= x >> 16. The same
 * seed and inputs give the same result.
 *   tensors    HOST array, read before the call returns. Pointers are aligned to their elements;
 *              tensors that are written share no memory with others
 *   state_bits 32: m and v are fp32. 8: codes, with the scale bytes in m_scale and v_scale
 *   lr_device  fp32 [1] device, or NULL: the learning rate is lr
 *   grad_norm  fp32 [1] device (moe_grad_clip's norm), or NULL. With it the gradients are multiplied
 *              by min(1, max_norm / (norm + 1e-6)) (max_norm +inf: by 1), and a norm that is not
 *              finite skips the step: nothing is written
 *   counters   int64 [2] device, zeroed by the caller before the first step: the steps done, and a
 *              count of the kernel's own. Calls that share them must not overlap
 * lr, decay and eps finite and >= 0, beta1 and beta2 in [0, 1), max_norm > 0. n in [0, 65536]. eps
 * is held in fp32, at least 2^-149 unless it is 0; with 0, elements whose v is 0 become m / 0. */
typedef struct {
  void *param;         /* param_dtype [numel], written                                        */
  float *master;       /* fp32 [numel] behind bf16 weights, written; NULL for fp32 weights    */
  const void *grad;    /* grad_dtype [numel]                                                  */
  void *m, *v;         /* [numel] states: fp32, or uint8 codes of m and of sqrt(v)            */
  uint8_t *m_scale;    /* [ceil(numel / 256)] scale bytes of 8-bit states, NULL otherwise     */
  uint8_t *v_scale;
  int64_t numel;       /* >= 0                                                                */
  int32_t param_dtype; /* moe_dtype_t; MOE_DT_BF16 needs a master                             */
  int32_t grad_dtype;  /* moe_dtype_t                                                         */
  float decay;         /* weight decay                                                        */
  int32_t reserved;    /* 0                                                                   */
} moe_adamw_tensor_t;
moe_status_t moe_adamw_step(int32_t n, const moe_adamw_tensor_t *tensors, int32_t state_bits,
                            double lr, const float *lr_device, double beta1, double beta2,
                            double eps, const float *grad_norm, float max_norm, uint64_t seed,
                            int64_t *counters, moe_stream_t stream);
/* The values that 8-bit states stand for: m and sqrt(v), bf16 [numel] each (four significant bits:
 * exact). m_out, v_out: HOST arrays of n device pointers, element-aligned. */
moe_status_t moe_adamw_moments(int32_t n, const moe_adamw_tensor_t *tensors, void *const *m_out,
                               void *const *v_out, moe_stream_t stream);

/* E4M3 with one fp32 scale for each block of 128 (the layout of block-scaled FP8 checkpoints):
 *   a = max(amax of the block, 2^-100),  s = a / 448,  code = E4M3(v * (448 / a)),
 * each step one IEEE fp32 operation, codes rounded to nearest even and saturating; the value
 * represented is code * s. Blocks at an edge are short. A NaN stays NaN; a block with an infinity
 * becomes NaN as a whole once multiplied by its (infinite) scale.
 *
 * Blocks of 1 x 128 (activations, gradients) of x bf16 [M, N], row stride ldx >= N:
 *   q_row e4m3 [M, N], row stride ld_qrow; s_row fp32 [ceil(N/128), M], row stride ld_srow
 *         (the scale of row m, block b at s_row[b * ld_srow + m])
 *   q_col e4m3 [N, M] = the transpose, blocks along M, row stride ld_qcol;
 *         s_col fp32 [ceil(M/128), N], row stride ld_scol
 * Either pair may be NULL. Both are made from one read of x. */
moe_status_t fp8_block_quantize_rows(const void *x, int64_t ldx, int64_t M, int64_t N,
                                     uint8_t *q_row, int64_t ld_qrow, float *s_row,
                                     int64_t ld_srow, uint8_t *q_col, int64_t ld_qcol,
                                     float *s_col, int64_t ld_scol, moe_stream_t stream);
/* Blocks of 128 x 128 (weights) of w bf16 [N, K], row stride ldw >= K:
 *   q  e4m3 [N, K], row stride ldq;   s  fp32 [ceil(N/128), ceil(K/128)]
 *   qt e4m3 [K, N] = the transpose (the same codes), row stride ldqt;
 *   st fp32 [ceil(K/128), ceil(N/128)]
 * qt and st may both be NULL. */
moe_status_t fp8_block_quantize_weight(const void *w, int64_t ldw, int64_t N, int64_t K,
                                       uint8_t *q, int64_t ldq, float *s, uint8_t *qt,
                                       int64_t ldqt, float *st, moe_stream_t stream);
/* C[m][n] = sum_b sa[b][m] * sb * sum_{k in block b} a[m][k] * bq[n][k], fp32 accumulation.
 *   a   e4m3 [M, K], row stride lda;  sa fp32 [ceil(K/128), M], row stride ld_sa
 *   b   e4m3 [N, K], row stride ldb;  b_scale 1: sb fp32 [ceil(N/128), ceil(K/128)] (128 x 128
 *       blocks, row stride ld_sb); b_scale 0: sb fp32 [ceil(K/128), N] (1 x 128 blocks, ld_sb)
 *   c   [M, N] of c_dtype (BF16 or FP32), row stride ldc
 * a, b 16-byte aligned with lda, ldb multiples of 16; sa (and sb for b_scale 0) 16-byte aligned
 * with ld_sa (ld_sb) a multiple of 4; sb 4-byte aligned otherwise. M, N < 2^31 - 256, K < 2^31 -
 * 256. A linear layer y = x w^T is (q_row of x) x (q of w); its input gradient (q_row of dy) x
 * (qt of w); its weight gradient (q_col of dy) x (q_col of x).
 * The product of two scales is formed in fp32 first: it should be a normal number (the blocks' amaxes
 * multiply to between 2.4e-33 and 6.8e43), or results lose bits, or overflow with it.
 *   err device int32 or NULL: MOE_DEVERR_TIMEOUT if a bounded wait inside gave up (sticky) */
moe_status_t fp8_block_gemm(const uint8_t *a, int64_t lda, const float *sa, int64_t ld_sa,
                            const uint8_t *b, int64_t ldb, const float *sb, int64_t ld_sb,
                            int32_t b_scale, void *c, int64_t ldc, int32_t c_dtype, int64_t M,
                            int64_t N, int64_t K, int32_t *err, moe_stream_t stream);

/* Enqueue a copy of the device error word into *host_code (pinned or pageable host int);
 * the value is valid once the stream has been synchronised. */
moe_status_t moe_get_error(const moe_layer_desc_t *desc, const void *ws, int32_t *host_code,
                           moe_stream_t stream);
/* Enqueue a reset of the device error word to MOE_DEVERR_NONE. */
moe_status_t moe_clear_error(const moe_layer_desc_t *desc, void *ws, moe_stream_t stream);

/* Failure-detection self-test (no counterpart on the pages; it exercises this library's own
 * bounded waits). Enqueues one kernel whose single barrier wait can never complete: the same
 * bounded wait the GEMM kernels use gives up after limit_ns nanoseconds (1 ms .. 10 s) and
 * writes MOE_DEVERR_TIMEOUT into *err (device int32; written only if it holds 0). The kernel
 * then returns normally, so the context stays usable; no fault, trap or endless loop is
 * involved. Returns MOE_ERR_INVALID_ARG for a NULL err or a limit outside the range. */
moe_status_t moe_selftest_wait_timeout(int32_t *err, uint64_t limit_ns, moe_stream_t stream);

/* Failure-detection self-test of a GEMM kernel itself (no counterpart on the pages). For a BF16
 * layer whose moe_route_permute (and forward) ran on ws, enqueues the FC2 forward grouped GEMM
 * (a_s x W2 -> the workspace's permuted output; w2 as for moe_grouped_mlp_fwd) with its TMA
 * producer issuing no loads. Every MMA and epilogue wait of the kernel then runs out after
 * limit_ns nanoseconds (1 ms .. 10 s): the CTA raises its abort flag, MOE_DEVERR_TIMEOUT goes
 * into the workspace error word (moe_get_error; moe_clear_error resets it), every role leaves
 * its loop, TMEM is freed and the kernel returns, so the context stays usable. The permuted
 * output in the workspace is left undefined until the next forward. Returns
 * MOE_ERR_UNSUPPORTED for a non-BF16 layer, MOE_ERR_INVALID_ARG for a bad description,
 * workspace, w2 or limit. */
moe_status_t moe_selftest_gemm_timeout(const moe_layer_desc_t *desc, void *ws, size_t ws_bytes,
                                       const void *w2, uint64_t limit_ns, moe_stream_t stream);

/* Number of SMs the persistent GEMM uses on the current device for this description
 * (device SM count minus sm_margin, at least 1). */
int32_t moe_gemm_ctas(const moe_layer_desc_t *desc);

/* Kernels this library enqueued on any stream since load (a monotonically increasing
 * host-side counter, for launch accounting). */
uint64_t moe_launch_count(void);

/* Kernel identifiers reported by the launch timeline. */
typedef enum {
  MOE_K_ROUTE_TOPK = 0,
  MOE_K_ASSIGN_ROWS = 1,
  MOE_K_GATHER_X = 2,
  MOE_K_GEMM_FC1_FPROP = 3,
  MOE_K_GEMM_FC2_FPROP = 4,
  MOE_K_COMBINE_Y = 5,
  MOE_K_GATHER_DY = 6,
  MOE_K_GEMM_FC2_DGRAD = 7,
  MOE_K_DPROB_REDUCE = 8,
  MOE_K_GEMM_FC2_WGRAD = 9,
  MOE_K_GEMM_FC1_DGRAD = 10,
  MOE_K_COMBINE_DX = 11,
  MOE_K_GEMM_FC1_WGRAD = 12,
  MOE_K_MXFP8_QUANTIZE = 13,
  MOE_K_PACK_FC1 = 14,
  MOE_K_EXTRAS_REDUCE = 15,
  MOE_K_NVFP4_AMAX = 16,
  MOE_K_NVFP4_QUANTIZE = 17,
  MOE_K_ROUTE_EXPORT = 18,
  MOE_K_ROUTER_LOSS = 19,
  MOE_K_ROUTER_GRAD = 20,
  MOE_K_LAYERNORM_FWD = 21,
  MOE_K_LAYERNORM_BWD = 22,
  MOE_K_LAYERNORM_REDUCE = 23,
  MOE_K_GRAD_NORM = 24,
  MOE_K_GRAD_SCALE = 25,
  MOE_K_FP8_QUANTIZE = 26,
  MOE_K_FP8_GEMM = 27,
  MOE_K_COUNT_IDS = 28,
  MOE_K_ROUTER_TOPK = 29,
  MOE_K_ROUTER_TOPK_GRAD = 30,
  MOE_K_RESIDUAL_NORM_FWD = 31,
  MOE_K_RESIDUAL_NORM_BWD = 32,
  MOE_K_RESIDUAL_NORM_REDUCE = 33,
  MOE_K_ADAMW = 34,
  MOE_K_ADAMW_MOMENTS = 35,
  MOE_K_COUNT = 36
} moe_kernel_id_t;

/* Launch timeline, for measurement. Between moe_timeline_begin and moe_timeline_end the
 * library records events[i] (caller-created cudaEvent_t handles, passed as void*) on the
 * launching stream right after its i-th kernel launch, for i < capacity, and remembers the
 * kernel's moe_kernel_id_t. Kernels of one stream run in order, so the elapsed time between
 * consecutive events is the duration of the later kernel. Process-wide; not thread-safe.
 * moe_timeline_end copies the ids into kernel_ids (capacity entries, may be NULL), stops
 * recording and returns how many events were recorded. */
moe_status_t moe_timeline_begin(void *const *events, int32_t capacity);
int32_t moe_timeline_end(int32_t *kernel_ids);

/* Human-readable message for the last host-side error of the calling thread. */
const char *moe_last_error_string(void);

#ifdef __cplusplus
}
#endif

#endif /* MOEGMM_H_ */
