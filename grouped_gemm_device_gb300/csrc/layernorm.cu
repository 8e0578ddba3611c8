// Layer norm over the last dimension, forward and backward (moe_layernorm_fwd /
// moe_layernorm_bwd in include/moegmm.h).
//
//   y = (x - mean) rstd gamma + beta;  h = (x - mean) rstd, u = dy gamma:
//   dx = rstd (u - mean_n(u) - h mean_n(u h));  dgamma = sum_m dy h;  dbeta = sum_m dy
//
// Bound by HBM: the forward reads and writes M N elements once, the backward reads x and dy and
// writes dx once. A row stays in registers between its statistics and its use, so the variance is
// taken about the mean (two passes over registers, not E[x^2] - mean^2). Statistics, sums and the
// weight-gradient partials are fp32.
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kMaxParts = 160;  // backward blocks at most: rows of the partial weight gradients

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

// VEC consecutive elements (VEC * sizeof(T) a multiple of 16 bytes, or VEC = 1) as fp32.
template <typename T, int VEC>
MOE_DEVICE void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = to_f(*p);
  } else {
    constexpr int W = VEC * sizeof(T) / 16;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint4 q = reinterpret_cast<const uint4*>(p)[w];
      const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
          v[8 * w + 2 * i] = bf16_lo(u[i]);
          v[8 * w + 2 * i + 1] = bf16_hi(u[i]);
        } else {
          v[4 * w + i] = __uint_as_float(u[i]);
        }
      }
    }
  }
}
template <typename T, int VEC>
MOE_DEVICE void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(v[0]);
  } else {
    constexpr int W = VEC * sizeof(T) / 16;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      uint4 q;
      if constexpr (sizeof(T) == 2)
        q = make_uint4(pack_bf16x2(v[8 * w], v[8 * w + 1]), pack_bf16x2(v[8 * w + 2], v[8 * w + 3]),
                       pack_bf16x2(v[8 * w + 4], v[8 * w + 5]),
                       pack_bf16x2(v[8 * w + 6], v[8 * w + 7]));
      else
        q = make_uint4(__float_as_uint(v[4 * w]), __float_as_uint(v[4 * w + 1]),
                       __float_as_uint(v[4 * w + 2]), __float_as_uint(v[4 * w + 3]));
      reinterpret_cast<uint4*>(p)[w] = q;
    }
  }
}

// Sums of a and b over the G threads of a row's group (G = 32, or a whole block of G threads;
// `sm` then holds 2 * 32 floats and may be reused after the next call's first barrier).
template <int G>
MOE_DEVICE void row_sum2(float& a, float& b, float* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
  }
  if constexpr (G > 32) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    __syncthreads();
    if (lane == 0) {
      sm[w] = a;
      sm[32 + w] = b;
    }
    __syncthreads();
    a = 0.f;
    b = 0.f;
#pragma unroll
    for (int i = 0; i < G / 32; ++i) {
      a += sm[i];
      b += sm[32 + i];
    }
  }
}

// G threads a row, PER vectors of VEC elements a thread: N <= G * PER * VEC.
template <typename XT, typename WT, int VEC, int G, int PER>
__global__ void __launch_bounds__(G < 128 ? 128 : G) ln_fwd_kernel(
    const XT* __restrict__ x, int64_t ldx, const WT* __restrict__ gamma,
    const WT* __restrict__ beta, XT* __restrict__ y, int64_t ldy, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, int64_t M, int N, float eps) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[64];
  constexpr int R = (G < 128 ? 128 : G) / G;  // rows a block
  const int t = threadIdx.x % G;
  const int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / G;
  if (G == 32 && row >= M) return;  // a block's rows are its warps; otherwise R = 1
  const XT* xr = x + row * ldx;
  float v[PER][VEC];
  float s = 0.f, unused = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (i * G + t) * VEC;
    if (c < N) {
      load_vec<XT, VEC>(xr + c, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s += v[i][j];
  row_sum2<G>(s, unused, sm);
  const float mean = s / (float)N;
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    if ((i * G + t) * VEC < N) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float d = v[i][j] - mean;
        q += d * d;
      }
    }
  row_sum2<G>(q, unused, sm);
  const float rstd = 1.0f / sqrtf(q / (float)N + eps);
  if (t == 0) {
    if (mean_out) mean_out[row] = mean;
    if (rstd_out) rstd_out[row] = rstd;
  }
  XT* yr = y + row * ldy;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (i * G + t) * VEC;
    if (c < N) {
      float gm[VEC], bt[VEC], o[VEC];
      if (gamma) load_vec<WT, VEC>(gamma + c, gm);
      if (beta) load_vec<WT, VEC>(beta + c, bt);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = (v[i][j] - mean) * rstd;
        o[j] = (gamma ? h * gm[j] : h) + (beta ? bt[j] : 0.f);
      }
      store_vec<XT, VEC>(yr + c, o);
    }
  }
}

// Rows longer than a block's registers: three passes over the row (the later two from L2).
template <typename XT, typename WT>
__global__ void __launch_bounds__(1024) ln_fwd_long_kernel(
    const XT* x, int64_t ldx, const WT* __restrict__ gamma, const WT* __restrict__ beta, XT* y,
    int64_t ldy, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t M, int64_t N,
    float eps) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[64];
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const XT* xr = x + row * ldx;
    float s = 0.f, unused = 0.f, q = 0.f;
    for (int64_t c = threadIdx.x; c < N; c += 1024) s += to_f(xr[c]);
    row_sum2<1024>(s, unused, sm);
    const float mean = s / (float)N;
    for (int64_t c = threadIdx.x; c < N; c += 1024) {
      const float d = to_f(xr[c]) - mean;
      q += d * d;
    }
    row_sum2<1024>(q, unused, sm);
    const float rstd = 1.0f / sqrtf(q / (float)N + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
    for (int64_t c = threadIdx.x; c < N; c += 1024) {
      const float h = (to_f(xr[c]) - mean) * rstd;
      y[row * ldy + c] = from_f<XT>((gamma ? h * to_f(gamma[c]) : h) + (beta ? to_f(beta[c]) : 0.f));
    }
  }
}

// One block walks rows blockIdx, blockIdx + grid, ...; a thread owns the same PER * VEC columns
// of every row and keeps their dgamma and dbeta sums in registers until the end.
template <typename XT, typename WT, int VEC, int G, int PER>
__global__ void __launch_bounds__(G) ln_bwd_kernel(
    const XT* dy, int64_t lddy, const XT* x, int64_t ldx, const WT* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, XT* dx, int64_t lddx,
    float* __restrict__ part, int64_t M, int N) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[64];
  const int t = threadIdx.x;
  float dg[PER][VEC], db[PER][VEC];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const float mu = mean[row], rs = rstd[row];
    float h[PER][VEC], u[PER][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC;
      if (c < N) {
        float gm[VEC];
        load_vec<XT, VEC>(x + row * ldx + c, h[i]);
        load_vec<XT, VEC>(dy + row * lddy + c, u[i]);
        if (gamma) load_vec<WT, VEC>(gamma + c, gm);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          h[i][j] = (h[i][j] - mu) * rs;
          dg[i][j] += u[i][j] * h[i][j];
          db[i][j] += u[i][j];
          if (gamma) u[i][j] *= gm[j];
          s1 += u[i][j];
          s2 += u[i][j] * h[i][j];
        }
      }
    }
    row_sum2<G>(s1, s2, sm);
    s1 /= (float)N;
    s2 /= (float)N;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC;
      if (c < N) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = rs * (u[i][j] - s1 - h[i][j] * s2);
        store_vec<XT, VEC>(dx + row * lddx + c, o);
      }
    }
  }
  if (!part) return;
  float* pg = part + (int64_t)blockIdx.x * 2 * N;
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = (i * G + t) * VEC + j;
      if (c < N) {
        pg[c] = dg[i][j];
        pg[N + c] = db[i][j];
      }
    }
}

// Longer rows: the weight gradients' partials first (dx may be dy or x), then dx.
template <typename XT>
__global__ void __launch_bounds__(256) ln_bwd_cols_long_kernel(
    const XT* dy, int64_t lddy, const XT* x, int64_t ldx, const float* __restrict__ mean,
    const float* __restrict__ rstd, float* __restrict__ part, int64_t M, int64_t N) {
  MOE_GRIDDEP_ENTRY();
  float* pg = part + (int64_t)blockIdx.x * 2 * N;
  for (int64_t c = threadIdx.x; c < N; c += 256) {
    float dg = 0.f, db = 0.f;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
      const float d = to_f(dy[row * lddy + c]);
      dg += d * ((to_f(x[row * ldx + c]) - mean[row]) * rstd[row]);
      db += d;
    }
    pg[c] = dg;
    pg[N + c] = db;
  }
}
template <typename XT, typename WT>
__global__ void __launch_bounds__(1024) ln_bwd_rows_long_kernel(
    const XT* dy, int64_t lddy, const XT* x, int64_t ldx, const WT* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, XT* dx, int64_t lddx,
    int64_t M, int64_t N) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[64];
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const float mu = mean[row], rs = rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < N; c += 1024) {
      const float d = to_f(dy[row * lddy + c]);
      const float u = gamma ? d * to_f(gamma[c]) : d;
      s1 += u;
      s2 += u * ((to_f(x[row * ldx + c]) - mu) * rs);
    }
    row_sum2<1024>(s1, s2, sm);
    s1 /= (float)N;
    s2 /= (float)N;
    for (int64_t c = threadIdx.x; c < N; c += 1024) {
      const float d = to_f(dy[row * lddy + c]);
      const float u = gamma ? d * to_f(gamma[c]) : d;
      const float h = (to_f(x[row * ldx + c]) - mu) * rs;
      dx[row * lddx + c] = from_f<XT>(rs * (u - s1 - h * s2));
    }
  }
}

// dgamma[c] (columns [0, N)) and dbeta (columns [N, 2N)) = sum of the blocks' partials. A warp
// sums every eighth partial of 32 columns; the eight sums are added in order.
template <typename WT>
__global__ void __launch_bounds__(256) ln_colsum_kernel(const float* __restrict__ part, int nparts,
                                                        int64_t N, WT* __restrict__ dgamma,
                                                        WT* __restrict__ dbeta) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[8][32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * N)
    for (int b = w; b < nparts; b += 8) s += part[(int64_t)b * 2 * N + c];
  sm[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < 2 * N) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm[i][lane];
    if (c < N) {
      if (dgamma) dgamma[c] = from_f<WT>(s);
    } else if (dbeta) {
      dbeta[c - N] = from_f<WT>(s);
    }
  }
}

bool aligned_to(const void* p, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0;
}

struct LnArgs {
  const void *x, *dy, *gamma, *beta;
  void *y, *dx;
  int64_t ldx, ldy, lddy, lddx;
  float *mean, *rstd;
  int64_t M, N;
  float eps;
  float* part;
  int nparts;
  cudaStream_t s;
};

template <typename XT, typename WT, int VEC, int G, int PER>
void fwd_launch(const LnArgs& a) {
  constexpr int B = G < 128 ? 128 : G;
  const int64_t blocks = (a.M + B / G - 1) / (B / G);
  ln_fwd_kernel<XT, WT, VEC, G, PER><<<(unsigned)blocks, B, 0, a.s>>>(
      static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma),
      static_cast<const WT*>(a.beta), static_cast<XT*>(a.y), a.ldy, a.mean, a.rstd, a.M, (int)a.N,
      a.eps);
}

template <typename XT, typename WT>
void fwd_typed(const LnArgs& a) {
  constexpr int V = 16 / sizeof(XT);
  const bool vec = a.N % V == 0 && a.ldx % V == 0 && a.ldy % V == 0 && aligned_to(a.x, 16) &&
                   aligned_to(a.y, 16) && aligned_to(a.gamma, 16) && aligned_to(a.beta, 16);
  const int64_t N = a.N;
  if (vec) {
    if (N <= 32 * V) return fwd_launch<XT, WT, V, 32, 1>(a);
    if (N <= 32 * 4 * V) return fwd_launch<XT, WT, V, 32, 4>(a);
    if (N <= 256 * 2 * V) return fwd_launch<XT, WT, V, 256, 2>(a);
    if (N <= 512 * 4 * V) return fwd_launch<XT, WT, V, 512, 4>(a);
  } else {
    if (N <= 32 * 8) return fwd_launch<XT, WT, 1, 32, 8>(a);
    if (N <= 256 * 8) return fwd_launch<XT, WT, 1, 256, 8>(a);
    if (N <= 512 * 32) return fwd_launch<XT, WT, 1, 512, 32>(a);
  }
  const int grid = (int)std::min<int64_t>(a.M, (int64_t)std::max(device_sms(), 1) * 2);
  ln_fwd_long_kernel<XT, WT><<<grid, 1024, 0, a.s>>>(
      static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma),
      static_cast<const WT*>(a.beta), static_cast<XT*>(a.y), a.ldy, a.mean, a.rstd, a.M, a.N,
      a.eps);
}

int bwd_parts(int64_t M) {
  const int most = std::min(std::max(device_sms(), 1), kMaxParts);
  return (int)std::max<int64_t>(1, std::min<int64_t>(M, most));
}

template <typename XT, typename WT, int VEC, int G, int PER>
void bwd_launch(const LnArgs& a) {
  ln_bwd_kernel<XT, WT, VEC, G, PER><<<a.nparts, G, 0, a.s>>>(
      static_cast<const XT*>(a.dy), a.lddy, static_cast<const XT*>(a.x), a.ldx,
      static_cast<const WT*>(a.gamma), a.mean, a.rstd, static_cast<XT*>(a.dx), a.lddx, a.part, a.M,
      (int)a.N);
}

template <typename XT, typename WT>
void bwd_typed(const LnArgs& a) {
  constexpr int V = 16 / sizeof(XT);
  const bool vec = a.N % V == 0 && a.ldx % V == 0 && a.lddy % V == 0 && a.lddx % V == 0 &&
                   aligned_to(a.x, 16) && aligned_to(a.dy, 16) && aligned_to(a.dx, 16) &&
                   aligned_to(a.gamma, 16);
  const int64_t N = a.N;
  if (vec) {
    if (N <= 32 * V) return bwd_launch<XT, WT, V, 32, 1>(a);
    if (N <= 256 * V) return bwd_launch<XT, WT, V, 256, 1>(a);
    if (N <= 512 * 2 * V) return bwd_launch<XT, WT, V, 512, 2>(a);
    if (N <= 512 * 4 * V) return bwd_launch<XT, WT, V, 512, 4>(a);
  } else {
    if (N <= 32 * 8) return bwd_launch<XT, WT, 1, 32, 8>(a);
    if (N <= 512 * 8) return bwd_launch<XT, WT, 1, 512, 8>(a);
    if (N <= 512 * 32) return bwd_launch<XT, WT, 1, 512, 32>(a);
  }
  if (a.part) {
    ln_bwd_cols_long_kernel<XT><<<a.nparts, 256, 0, a.s>>>(
        static_cast<const XT*>(a.dy), a.lddy, static_cast<const XT*>(a.x), a.ldx, a.mean, a.rstd,
        a.part, a.M, a.N);
    count_launch(a.s, MOE_K_LAYERNORM_BWD);
  }
  const int grid = (int)std::min<int64_t>(a.M, (int64_t)std::max(device_sms(), 1) * 2);
  ln_bwd_rows_long_kernel<XT, WT><<<grid, 1024, 0, a.s>>>(
      static_cast<const XT*>(a.dy), a.lddy, static_cast<const XT*>(a.x), a.ldx,
      static_cast<const WT*>(a.gamma), a.mean, a.rstd, static_cast<XT*>(a.dx), a.lddx, a.M, a.N);
}

moe_status_t check_types(int64_t M, int64_t N, int32_t xd, int32_t wd) {
  if (M < 0 || N < 1) return fail(MOE_ERR_INVALID_ARG, "M must be >= 0 and N >= 1");
  if (N > INT32_MAX || M > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "M or N too large");
  if ((xd != MOE_DT_BF16 && xd != MOE_DT_FP32) || (wd != MOE_DT_BF16 && wd != MOE_DT_FP32))
    return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  if (xd == MOE_DT_FP32 && wd == MOE_DT_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "fp32 rows take fp32 weights");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_layernorm_fwd(const void* x, int64_t ldx, const void* gamma, const void* beta,
                               void* y, int64_t ldy, float* mean, float* rstd, int64_t M,
                               int64_t N, float eps, int32_t x_dtype, int32_t w_dtype,
                               moe_stream_t stream) {
  moe_status_t st = check_types(M, N, x_dtype, w_dtype);
  if (st != MOE_OK) return st;
  if (ldx < N || ldy < N) return fail(MOE_ERR_INVALID_ARG, "row strides must be >= N");
  if (!(eps >= 0.f)) return fail(MOE_ERR_INVALID_ARG, "eps must be >= 0");
  if (M == 0) return MOE_OK;
  if (!x || !y) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  const int xb = x_dtype == MOE_DT_BF16 ? 2 : 4, wb = w_dtype == MOE_DT_BF16 ? 2 : 4;
  if (!aligned_to(x, xb) || !aligned_to(y, xb) || !aligned_to(gamma, wb) ||
      !aligned_to(beta, wb) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  LnArgs a = {};
  a.x = x; a.ldx = ldx; a.gamma = gamma; a.beta = beta; a.y = y; a.ldy = ldy;
  a.mean = mean; a.rstd = rstd; a.M = M; a.N = N; a.eps = eps;
  a.s = reinterpret_cast<cudaStream_t>(stream);
  if (x_dtype == MOE_DT_FP32) fwd_typed<float, float>(a);
  else if (w_dtype == MOE_DT_FP32) fwd_typed<__nv_bfloat16, float>(a);
  else fwd_typed<__nv_bfloat16, __nv_bfloat16>(a);
  count_launch(a.s, MOE_K_LAYERNORM_FWD);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "layernorm forward launch");
  return MOE_OK;
}

size_t moe_layernorm_workspace(int64_t M, int64_t N) {
  if (M < 0 || N < 1 || M > INT32_MAX || N > INT32_MAX) {
    fail(MOE_ERR_INVALID_ARG, "M must be in [0, 2^31) and N in [1, 2^31)");
    return 0;
  }
  return (size_t)std::max<int64_t>(1, std::min<int64_t>(M, kMaxParts)) * 2 * N * sizeof(float);
}

moe_status_t moe_layernorm_bwd(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                               const void* gamma, const float* mean, const float* rstd, void* dx,
                               int64_t lddx, void* dgamma, void* dbeta, int64_t M, int64_t N,
                               int32_t x_dtype, int32_t w_dtype, void* ws, size_t ws_bytes,
                               moe_stream_t stream) {
  moe_status_t st = check_types(M, N, x_dtype, w_dtype);
  if (st != MOE_OK) return st;
  if (ldx < N || lddy < N || lddx < N)
    return fail(MOE_ERR_INVALID_ARG, "row strides must be >= N");
  const bool weights = dgamma || dbeta;
  if (M > 0 && (!dy || !x || !mean || !rstd || !dx))
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  const int xb = x_dtype == MOE_DT_BF16 ? 2 : 4, wb = w_dtype == MOE_DT_BF16 ? 2 : 4;
  if (!aligned_to(x, xb) || !aligned_to(dy, xb) || !aligned_to(dx, xb) || !aligned_to(gamma, wb) ||
      !aligned_to(dgamma, wb) || !aligned_to(dbeta, wb) || !aligned_to(mean, 4) ||
      !aligned_to(rstd, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (weights) {
    if (!ws || !aligned_to(ws, 16))
      return fail(MOE_ERR_INVALID_ARG, "ws must be non-NULL and 16-byte aligned");
    if (ws_bytes < moe_layernorm_workspace(M, N))
      return fail(MOE_ERR_WORKSPACE, "ws_bytes=%zu < required %zu", ws_bytes,
                  moe_layernorm_workspace(M, N));
  }
  if (M == 0 && !weights) return MOE_OK;
  LnArgs a = {};
  a.x = x; a.ldx = ldx; a.dy = dy; a.lddy = lddy; a.gamma = gamma; a.dx = dx; a.lddx = lddx;
  a.mean = const_cast<float*>(mean); a.rstd = const_cast<float*>(rstd);
  a.M = M; a.N = N;
  a.part = weights ? static_cast<float*>(ws) : nullptr;
  a.nparts = bwd_parts(M);
  a.s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (M > 0) {
    if (x_dtype == MOE_DT_FP32) bwd_typed<float, float>(a);
    else if (w_dtype == MOE_DT_FP32) bwd_typed<__nv_bfloat16, float>(a);
    else bwd_typed<__nv_bfloat16, __nv_bfloat16>(a);
    count_launch(a.s, MOE_K_LAYERNORM_BWD);
    e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e, "layernorm backward launch");
  } else {
    a.nparts = 0;  // no rows: the sums are zero
  }
  if (weights) {
    const unsigned grid = (unsigned)((2 * N + 31) / 32);
    if (w_dtype == MOE_DT_FP32)
      e = launch_chained(ln_colsum_kernel<float>, grid, 256, 0, a.s, (const float*)a.part,
                         a.nparts, N, static_cast<float*>(dgamma), static_cast<float*>(dbeta));
    else
      e = launch_chained(ln_colsum_kernel<__nv_bfloat16>, grid, 256, 0, a.s,
                         (const float*)a.part, a.nparts, N, static_cast<__nv_bfloat16*>(dgamma),
                         static_cast<__nv_bfloat16*>(dbeta));
    count_launch(a.s, MOE_K_LAYERNORM_REDUCE);
    if (e != cudaSuccess) return cuda_fail(e, "layernorm reduction launch");
  }
  return MOE_OK;
}

}  // extern "C"
