// The residual stream around a block and its two root-mean-square norms, forward and backward
// (moe_residual_norm_fwd / moe_residual_norm_bwd in include/moegmm.h).
//
//   u = wp o rp,  x' = x + s g u,  h = w x' r;       rp, r = 1 / sqrt(mean(.^2) + eps)
//   y = x' r, z = o rp:  dx = dx' + r (dh w - y mean(dh w y));  e = dx wp
//   do = s g rp (e - z mean(e z));  dg = s sum(e z);  dwp = sum_m s g dx z;  dw = sum_m dh y
//
// Bound by HBM: the forward reads x and o and writes x' and h, the backward reads dh, dx', x' and o
// and writes dx and do.
#include "kernels.cuh"

namespace moe {
namespace {

template <typename T>
MOE_DEVICE float to_f(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}
template <typename T>
MOE_DEVICE T from_f(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}
// A norm's weight: bf16, fp32 or none (1).
struct Weight {
  const void* p;
  int fp32;
};
MOE_DEVICE float weight_at(const Weight& w, int64_t c) {
  if (!w.p) return 1.0f;
  return w.fp32 ? static_cast<const float*>(w.p)[c]
                : __bfloat162float(static_cast<const __nv_bfloat16*>(w.p)[c]);
}

// Sum over a block of 1024 threads, the same in each. `sm` must not be in use by a call less than
// one barrier ago.
MOE_DEVICE float block_sum(float a, float (&sm)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  const int lane = threadIdx.x & 31;
  if (lane == 0) sm[threadIdx.x >> 5] = a;
  __syncthreads();
  a = sm[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  return a;
}

struct FwdArgs {
  const void *x, *o;
  void *xn, *h;
  int64_t ldx, ldo, ldxn, ldh, M, N;
  Weight wp, w;
  const float* gate;
  float *rstd_post, *rstd;
  float scale, eps;
  int post;
};

// Any length, stride and place: a block a row, element by element, the row once for each sum and
// once for each result (the later ones from L2).
template <typename XT, typename OT>
__global__ void __launch_bounds__(1024) rn_fwd_any_kernel(const FwdArgs a) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[2][32];
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    const OT* o = static_cast<const OT*>(a.o) + row * a.ldo;
    XT* xn = static_cast<XT*>(a.xn) + row * a.ldxn;
    float rp = 1.0f;
    if (a.post) {
      float s = 0.f;
      for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
        const float v = to_f(o[c]);
        s += v * v;
      }
      rp = 1.0f / sqrtf(block_sum(s, sm[0]) / (float)a.N + a.eps);
      if (threadIdx.x == 0 && a.rstd_post) a.rstd_post[row] = rp;
    }
    const float q = a.gate ? a.scale * a.gate[row] : a.scale;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
      XT v = x[c];
      if (a.o) {
        const float z = a.post ? to_f(o[c]) * rp : to_f(o[c]);
        v = from_f<XT>(to_f(v) + q * (z * weight_at(a.wp, c)));
        xn[c] = v;
      }
      s += to_f(v) * to_f(v);
    }
    if (a.h) {
      const float r = 1.0f / sqrtf(block_sum(s, sm[1]) / (float)a.N + a.eps);
      if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
      const XT* y = a.o ? xn : x;
      for (int64_t c = threadIdx.x; c < a.N; c += 1024)
        static_cast<OT*>(a.h)[row * a.ldh + c] = from_f<OT>(to_f(y[c]) * r * weight_at(a.w, c));
    }
    __syncthreads();  // the sums' places are used again
  }
}

struct BwdArgs {
  const void *dh, *dxn, *xn, *o;
  void *dx, *d_o;
  int64_t lddh, lddxn, ldxn, ldo, lddx, lddo, M, N;
  Weight wp, w;
  const float *gate, *rstd_post, *rstd;
  float* d_gate;
  float scale;
  int post;
  float* part;  // [blocks][2][N]: dw, dwp
};

template <typename XT, typename OT>
__global__ void __launch_bounds__(1024) rn_bwd_any_kernel(const BwdArgs a) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[2][32];
  float* part = a.part ? a.part + (int64_t)blockIdx.x * 2 * a.N : nullptr;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const OT* dh = static_cast<const OT*>(a.dh) + row * a.lddh;
    const XT* dxn = static_cast<const XT*>(a.dxn) + row * a.lddxn;
    const XT* xn = static_cast<const XT*>(a.xn) + row * a.ldxn;
    const OT* o = static_cast<const OT*>(a.o) + row * a.ldo;
    const float r = a.dh ? a.rstd[row] : 0.f, rp = a.post ? a.rstd_post[row] : 1.0f;
    const float q = a.gate ? a.scale * a.gate[row] : a.scale;
    float c1 = 0.f;
    if (a.dh) {
      for (int64_t c = threadIdx.x; c < a.N; c += 1024)
        c1 += to_f(dh[c]) * weight_at(a.w, c) * (to_f(xn[c]) * r);
      c1 = block_sum(c1, sm[0]) / (float)a.N;
    }
    auto grad = [&](int64_t c) {
      float d = a.dxn ? to_f(dxn[c]) : 0.f;
      if (a.dh) d += r * (to_f(dh[c]) * weight_at(a.w, c) - to_f(xn[c]) * r * c1);
      return d;
    };
    float dot = 0.f;
    if (a.o && (a.post || a.d_gate)) {
      for (int64_t c = threadIdx.x; c < a.N; c += 1024)
        dot += grad(c) * weight_at(a.wp, c) * (to_f(o[c]) * rp);
      dot = block_sum(dot, sm[1]);
      if (threadIdx.x == 0 && a.d_gate) a.d_gate[row] = a.scale * dot;
    }
    const float c2 = a.post ? dot / (float)a.N : 0.f;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
      const float d = grad(c);
      const float y = a.dh ? to_f(xn[c]) * r : 0.f, dw = a.dh ? to_f(dh[c]) * y : 0.f;
      const float z = a.o ? to_f(o[c]) * rp : 0.f, dwp = q * d * z;
      if (part) {  // column c belongs to this thread in every row
        part[c] = first ? dw : part[c] + dw;
        part[a.N + c] = first ? dwp : part[a.N + c] + dwp;
      }
      if (a.dx) static_cast<XT*>(a.dx)[row * a.lddx + c] = from_f<XT>(d);
      if (a.d_o)
        static_cast<OT*>(a.d_o)[row * a.lddo + c] =
            from_f<OT>(q * rp * (d * weight_at(a.wp, c) - z * c2));
    }
    first = false;
    __syncthreads();
  }
}

// dw (columns [0, N)) and dwp (columns [N, 2 N)) = sum of the blocks' partials in a fixed order.
template <typename WT>
__global__ void __launch_bounds__(1024) rn_colsum_kernel(const float* __restrict__ part,
                                                         int nparts, int64_t N,
                                                         WT* __restrict__ dw,
                                                         WT* __restrict__ dwp) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * N)
    for (int b = w; b < nparts; b += 32) s += part[(int64_t)b * 2 * N + c];
  sm[w][lane] = s;
  __syncthreads();
  s = sm[lane][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int64_t col = (int64_t)blockIdx.x * 32 + w;
  if (lane == 0 && col < 2 * N) {
    if (col < N) {
      if (dw) dw[col] = from_f<WT>(s);
    } else if (dwp) {
      dwp[col - N] = from_f<WT>(s);
    }
  }
}

constexpr int64_t kMaxParts = 480;  // rows of partial weight gradients

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int size_of(int32_t dtype) { return dtype == MOE_DT_FP32 ? 4 : 2; }

// Calls fn with values of the stream's and the branch's type.
template <class F>
cudaError_t typed(int32_t xd, int32_t od, F&& fn) {
  if (xd == MOE_DT_BF16) return fn(__nv_bfloat16(), __nv_bfloat16());
  if (od == MOE_DT_BF16) return fn(float(), __nv_bfloat16());
  return fn(float(), float());
}

moe_status_t check_types(int64_t M, int64_t N, int32_t xd, int32_t od, int32_t wd) {
  if (M < 0 || N < 1) return fail(MOE_ERR_INVALID_ARG, "M must be >= 0 and N >= 1");
  if (N > INT32_MAX || M > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "M or N too large");
  for (int32_t d : {xd, od, wd})
    if (d != MOE_DT_BF16 && d != MOE_DT_FP32) return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  if (xd == MOE_DT_BF16 && od == MOE_DT_FP32)
    return fail(MOE_ERR_UNSUPPORTED, "a bf16 stream takes bf16 branches");
  if (od == MOE_DT_FP32 && wd == MOE_DT_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "fp32 branches take fp32 weights");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_residual_norm_fwd(const void* x, int64_t ldx, const void* o, int64_t ldo,
                                   const void* post_weight, const float* gate,
                                   const void* weight, void* x_new, int64_t ldxn, void* h,
                                   int64_t ldh, float* rstd_post, float* rstd, int64_t M,
                                   int64_t N, float scale, int32_t post_norm, float eps,
                                   int32_t x_dtype, int32_t o_dtype, int32_t w_dtype,
                                   moe_stream_t stream) {
  moe_status_t st = check_types(M, N, x_dtype, o_dtype, w_dtype);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f)) return fail(MOE_ERR_INVALID_ARG, "eps must be >= 0");
  if (M == 0) return MOE_OK;  // empty tensors' pointers may be NULL
  if ((o != nullptr) != (x_new != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "o and x_new go together");
  if (!o && (post_weight || gate || post_norm))
    return fail(MOE_ERR_INVALID_ARG, "post_weight, gate and post_norm need a branch");
  if (!h && weight) return fail(MOE_ERR_INVALID_ARG, "weight needs h");
  if (!o && !h) return fail(MOE_ERR_INVALID_ARG, "neither a branch nor h");
  if (ldx < N || (o && (ldo < N || ldxn < N)) || (h && ldh < N))
    return fail(MOE_ERR_INVALID_ARG, "row strides must be >= N");
  if (x_new == x && x_new && ldxn != ldx)
    return fail(MOE_ERR_INVALID_ARG, "x_new is x, with another row stride");
  if (h == o && h && ldh != ldo)
    return fail(MOE_ERR_INVALID_ARG, "h is o, with another row stride");
  const int xb = size_of(x_dtype), ob = size_of(o_dtype), wb = size_of(w_dtype);
  if (!on(x, xb) || !on(x_new, xb) || !on(o, ob) || !on(h, ob) || !on(post_weight, wb) ||
      !on(weight, wb) || !on(gate, 4) || !on(rstd_post, 4) || !on(rstd, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (!x) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  const int w32 = w_dtype == MOE_DT_FP32;
  const FwdArgs a = {x, o, x_new, h, ldx, ldo, ldxn, ldh, M, N, {post_weight, w32}, {weight, w32},
                     gate, rstd_post, rstd, scale, eps, post_norm != 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = (int)std::min<int64_t>(M, (int64_t)std::max(device_sms(), 1) * 2);
  const cudaError_t e = typed(x_dtype, o_dtype, [&](auto xt, auto ot) {
    return launch_pdl(rn_fwd_any_kernel<decltype(xt), decltype(ot)>, grid, 1024, 0, s, 1, a);
  });
  count_launch(s, MOE_K_RESIDUAL_NORM_FWD);
  if (e != cudaSuccess) return cuda_fail(e, "residual norm forward launch");
  return MOE_OK;
}

size_t moe_residual_norm_workspace(int64_t M, int64_t N) {
  if (M < 0 || N < 1 || M > INT32_MAX || N > INT32_MAX) {
    fail(MOE_ERR_INVALID_ARG, "M must be in [0, 2^31) and N in [1, 2^31)");
    return 0;
  }
  return (size_t)std::max<int64_t>(1, std::min<int64_t>(M, kMaxParts)) * 2 * (N + 8) *
         sizeof(float);
}

moe_status_t moe_residual_norm_bwd(const void* dh, int64_t lddh, const void* dx_new,
                                   int64_t lddxn, const void* x_new, int64_t ldxn, const void* o,
                                   int64_t ldo, const void* post_weight, const float* gate,
                                   const void* weight, const float* rstd_post, const float* rstd,
                                   void* dx, int64_t lddx, void* d_o, int64_t lddo,
                                   void* d_post_weight, void* d_weight, float* d_gate, int64_t M,
                                   int64_t N, float scale, int32_t post_norm, int32_t x_dtype,
                                   int32_t o_dtype, int32_t w_dtype, void* ws, size_t ws_bytes,
                                   moe_stream_t stream) {
  moe_status_t st = check_types(M, N, x_dtype, o_dtype, w_dtype);
  if (st != MOE_OK) return st;
  const bool weights = d_weight || d_post_weight;
  if (M > 0) {  // empty tensors' pointers may be NULL
    if (!dh && !dx_new) return fail(MOE_ERR_INVALID_ARG, "neither dh nor dx_new");
    if (!dh && (weight || d_weight))
      return fail(MOE_ERR_INVALID_ARG, "weight and d_weight need dh");
    if (dh && (!x_new || !rstd)) return fail(MOE_ERR_INVALID_ARG, "dh needs x_new and rstd");
    if (!o && (d_o || d_post_weight || d_gate || post_weight || gate || post_norm))
      return fail(MOE_ERR_INVALID_ARG, "post_weight, gate, post_norm and gradients need a branch");
    if (post_norm && !rstd_post) return fail(MOE_ERR_INVALID_ARG, "post_norm needs rstd_post");
    if (d_gate && !gate) return fail(MOE_ERR_INVALID_ARG, "d_gate needs a gate");
    if (!dx && !d_o && !weights && !d_gate) return fail(MOE_ERR_INVALID_ARG, "nothing to write");
    if ((dh && (lddh < N || ldxn < N)) || (dx_new && lddxn < N) || (o && ldo < N) ||
        (dx && lddx < N) || (d_o && lddo < N))
      return fail(MOE_ERR_INVALID_ARG, "row strides must be >= N");
    if ((dx && dx == dx_new && lddx != lddxn) || (d_o && d_o == dh && lddo != lddh) ||
        (d_o && d_o == o && lddo != ldo))
      return fail(MOE_ERR_INVALID_ARG, "an output is an input, with another row stride");
  }
  if (d_post_weight && !post_weight)
    return fail(MOE_ERR_INVALID_ARG, "d_post_weight needs post_weight");
  const int xb = size_of(x_dtype), ob = size_of(o_dtype), wb = size_of(w_dtype);
  if (!on(dh, ob) || !on(dx_new, xb) || !on(x_new, xb) || !on(o, ob) || !on(dx, xb) ||
      !on(d_o, ob) || !on(post_weight, wb) || !on(weight, wb) || !on(d_post_weight, wb) ||
      !on(d_weight, wb) || !on(gate, 4) || !on(rstd_post, 4) || !on(rstd, 4) || !on(d_gate, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (weights) {
    if (!ws || !on(ws, 16))
      return fail(MOE_ERR_INVALID_ARG, "ws must be non-NULL and 16-byte aligned");
    if (ws_bytes < moe_residual_norm_workspace(M, N))
      return fail(MOE_ERR_WORKSPACE, "ws_bytes=%zu < required %zu", ws_bytes,
                  moe_residual_norm_workspace(M, N));
  }
  if (M == 0 && !weights) return MOE_OK;
  const int w32 = w_dtype == MOE_DT_FP32;
  float* part = weights ? static_cast<float*>(ws) : nullptr;
  const BwdArgs a = {dh, dx_new, x_new, o, dx, d_o, lddh, lddxn, ldxn, ldo, lddx, lddo, M, N,
                     {post_weight, w32}, {weight, w32}, gate, rstd_post, rstd, d_gate, scale,
                     post_norm != 0, part};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const int nparts = (int)std::min<int64_t>(
      M, std::min<int64_t>((int64_t)std::max(device_sms(), 1) * 2, kMaxParts));
  if (M > 0) {
    e = typed(x_dtype, o_dtype, [&](auto xt, auto ot) {
      return launch_pdl(rn_bwd_any_kernel<decltype(xt), decltype(ot)>, nparts, 1024, 0, s, 1, a);
    });
    count_launch(s, MOE_K_RESIDUAL_NORM_BWD);
    if (e != cudaSuccess) return cuda_fail(e, "residual norm backward launch");
  }  // no rows: no partials, the sums are zero
  if (weights) {
    const unsigned grid = (unsigned)((2 * N + 31) / 32);
    if (w32)
      e = launch_pdl(rn_colsum_kernel<float>, grid, 1024, 0, s, 1, (const float*)part, nparts, N,
                     static_cast<float*>(d_weight), static_cast<float*>(d_post_weight));
    else
      e = launch_pdl(rn_colsum_kernel<__nv_bfloat16>, grid, 1024, 0, s, 1, (const float*)part,
                     nparts, N, static_cast<__nv_bfloat16*>(d_weight),
                     static_cast<__nv_bfloat16*>(d_post_weight));
    count_launch(s, MOE_K_RESIDUAL_NORM_REDUCE);
    if (e != cudaSuccess) return cuda_fail(e, "residual norm reduction launch");
  }
  return MOE_OK;
}

}  // extern "C"
