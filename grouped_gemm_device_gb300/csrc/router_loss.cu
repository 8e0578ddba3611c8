// Load-balance loss of a top-k router, its per-expert counts, and the gradient of the router's
// logits (moe_router_loss_fwd / moe_router_loss_bwd in include/moegmm.h).
//
//   p = softmax(logits) over E;  P_e = mean over valid tokens of p_e;  f_e = E c_e / (k n)
//   loss = coef sum_e f_e P_e
//   d_logits = mask g coef/n p (f - <p, f>)  +  scatter_j w_j (d_j - <w, d>)
//
// Both passes stream the fp32 logits once and are bound by HBM (or, for a few thousand tokens,
// by the launches). A token's row is spread over L lanes of a warp (L the power of two that gives
// each lane one VEC-wide load where it can, so 32/L tokens share a warp), its softmax takes
// log2(L) shuffles twice, and nothing but the row's own E values is kept in registers.
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 256;  // partial rows the workspace holds

// One block's share: sum of p over its valid tokens and the pairs routed to the expert. Entry E
// holds the number of valid tokens in c.
struct Partial {
  float p;
  int c;
};

// Row of a token over the lanes of its group: value i*VEC + j of lane `sub` is expert
// (i*L + sub)*VEC + j. NaN and entries past E read as -inf (weight 0 unless the whole row is).
template <int VEC, int V>
MOE_DEVICE void load_row(const float* row, int E, int L, int sub, float (&v)[V * VEC]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (i * L + sub) * VEC;
    if constexpr (VEC == 4) {
      float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) q = __ldg(reinterpret_cast<const float4*>(row + e));  // E % 4 == 0
      v[4 * i] = q.x;
      v[4 * i + 1] = q.y;
      v[4 * i + 2] = q.z;
      v[4 * i + 3] = q.w;
    } else {
      v[i] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < V * VEC; ++i) v[i] = v[i] == v[i] ? v[i] : -INFINITY;
}

MOE_DEVICE float group_max(float x, int L) {
  for (int o = L >> 1; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}
MOE_DEVICE float group_sum(float x, int L) {
  for (int o = L >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// v <- softmax over the group; a value equal to the maximum weighs 1 (also an infinite one).
template <int VEC, int V>
MOE_DEVICE void softmax_row(float (&v)[V * VEC], int E, int L, int sub) {
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < V * VEC; ++i) m = fmaxf(m, v[i]);
  m = group_max(m, L);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      float& x = v[i * VEC + j];
      const bool in = (i * L + sub) * VEC + j < E;
      x = !in ? 0.f : x == m ? 1.0f : expf(x - m);
      s += x;
    }
  s = group_sum(s, L);
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < V * VEC; ++i) v[i] *= inv;
}

// The block's partials, or (one block) straight to the results.
MOE_DEVICE void finish_expert(int e, double p, int c, int n, int E, int k, float* mean_prob,
                              int32_t* counts, double& term) {
  const double mp = n > 0 ? p / n : 0.0;
  mean_prob[e] = (float)mp;
  counts[e] = c;
  if (n > 0) term += mp * ((double)E * c / ((double)k * n));
}

template <int VEC, int V>
__global__ void __launch_bounds__(kThreads) router_loss_kernel(
    const float* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, int T, int E, int k, int L, Partial* __restrict__ part) {
  MOE_GRIDDEP_ENTRY();
  __shared__ int hist[257];
  __shared__ float psum[kWarps][256];
  for (int i = threadIdx.x; i <= E; i += kThreads) hist[i] = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (L - 1), grp = lane / L, G = 32 / L;
  const int64_t stride = (int64_t)gridDim.x * kWarps * G;
  float acc[V * VEC];
#pragma unroll
  for (int i = 0; i < V * VEC; ++i) acc[i] = 0.f;
  int valid = 0;
  __syncthreads();
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * G; t0 < T; t0 += stride) {
    const int64_t t = t0 + grp;
    const bool live = t < T && (!mask || mask[t]);
    float v[V * VEC];
    load_row<VEC, V>(logits + (t < T ? t : t0) * ld, E, L, sub, v);
    softmax_row<VEC, V>(v, E, L, sub);
    if (live) {
#pragma unroll
      for (int i = 0; i < V * VEC; ++i) acc[i] += v[i];
      valid += sub == 0;
      for (int j = sub; j < k; j += L) {
        const int e = ids[t * k + j];
        if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
      }
    }
  }
  // the warp's token groups, then the block's warps, in a fixed order
#pragma unroll
  for (int i = 0; i < V * VEC; ++i)
    for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int e = (i * L + sub) * VEC + j;
        if (e < E) psum[warp][e] = acc[i * VEC + j];
      }
  }
  if (valid) atomicAdd(&hist[E], valid);
  __syncthreads();
  for (int e = threadIdx.x; e <= E; e += kThreads) {
    Partial o;
    o.c = hist[e];
    o.p = 0.f;
    if (e < E)
      for (int w = 0; w < kWarps; ++w) o.p += psum[w][e];
    part[(int64_t)blockIdx.x * (E + 1) + e] = o;
  }
}

// Sums the blocks' partials in block order and forms the loss (one block).
__global__ void __launch_bounds__(1024) router_loss_finish_kernel(
    const Partial* __restrict__ part, int nblk, int E, int k, float coef, float* loss,
    int32_t* counts, float* mean_prob, int32_t* n_valid) {
  MOE_GRIDDEP_ENTRY();
  __shared__ double sp[1024];
  __shared__ int sc[1024];
  __shared__ int s_n;
  __shared__ double s_term[32];
  // thread (g, e): every fourth block's entry of expert e (E <= 256); valid tokens separately
  const int g = threadIdx.x >> 8, e = threadIdx.x & 255;
  double p = 0.0;
  int c = 0;
  if (e < E)
    for (int b = g; b < nblk; b += 4) {
      const Partial q = part[(int64_t)b * (E + 1) + e];
      p += q.p;
      c += q.c;
    }
  sp[threadIdx.x] = p;
  sc[threadIdx.x] = c;
  if (threadIdx.x < 32) {
    int n = 0;
    for (int b = threadIdx.x; b < nblk; b += 32) n += part[(int64_t)b * (E + 1) + E].c;
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
    if (threadIdx.x == 0) s_n = n;
  }
  __syncthreads();
  const int n = s_n;
  double term = 0.0;
  if (threadIdx.x < E) {
    const int x = threadIdx.x;
    finish_expert(x, (sp[x] + sp[x + 256]) + (sp[x + 512] + sp[x + 768]),
                  sc[x] + sc[x + 256] + sc[x + 512] + sc[x + 768], n, E, k, mean_prob, counts,
                  term);
  }
  for (int o = 16; o > 0; o >>= 1) term += __shfl_xor_sync(0xFFFFFFFFu, term, o);
  if ((threadIdx.x & 31) == 0) s_term[threadIdx.x >> 5] = term;
  __syncthreads();
  if (threadIdx.x == 0) {
    double s = 0.0;
    for (int w = 0; w < 8; ++w) s += s_term[w];
    *loss = (float)((double)coef * s);
    *n_valid = n;
  }
}

template <int VEC, int V>
__global__ void __launch_bounds__(kThreads) router_grad_kernel(
    const float* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const float* __restrict__ w, const float* __restrict__ dw, const uint8_t* __restrict__ mask,
    int T, int E, int k, int L, float coef, const float* __restrict__ d_loss,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ n_valid,
    float* __restrict__ d, int64_t ldd) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float f[256];
  // the chosen probabilities' part of a warp's rows, added by slot and read back by expert
  __shared__ float chosen[kWarps][32 * 8];
  const int n = *n_valid;
  const float g = n > 0 ? (d_loss ? *d_loss : 1.0f) * coef / (float)n : 0.f;
  for (int e = threadIdx.x; e < 256; e += kThreads)
    f[e] = e < E && n > 0 ? (float)((double)E * counts[e] / ((double)k * n)) : 0.f;
  for (int i = threadIdx.x; i < kWarps * 32 * 8; i += kThreads) (&chosen[0][0])[i] = 0.f;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (L - 1), grp = lane / L, G = 32 / L;
  const int64_t stride = (int64_t)gridDim.x * kWarps * G;
  float* row_c = &chosen[warp][grp * L * V * VEC];  // G * L * V * VEC <= 256
  float fe[V * VEC];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int e = (i * L + sub) * VEC + j;
      fe[i * VEC + j] = e < E ? f[e] : 0.f;
    }
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * G; t0 < T; t0 += stride) {
    const int64_t t = t0 + grp;
    const bool in = t < T;
    float v[V * VEC];
    load_row<VEC, V>(logits + (in ? t : t0) * ld, E, L, sub, v);
    softmax_row<VEC, V>(v, E, L, sub);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V * VEC; ++i) s += v[i] * fe[i];
    s = group_sum(s, L);
    const float c = in && (!mask || mask[t]) ? g : 0.f;
    if (w) {
      float dot = 0.f;
      if (in)
        for (int j = sub; j < k; j += L) {
          const int e = ids[t * k + j];
          if (e >= 0 && e < E) dot += w[t * k + j] * dw[t * k + j];
        }
      dot = group_sum(dot, L);
      __syncwarp();
      if (in)
        for (int j = sub; j < k; j += L) {
          const int e = ids[t * k + j];
          if (e >= 0 && e < E) atomicAdd(&row_c[e], w[t * k + j] * (dw[t * k + j] - dot));
        }
      __syncwarp();
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (i * L + sub) * VEC;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int q = i * VEC + j;
        o[j] = c != 0.f ? c * v[q] * (fe[q] - s) : 0.f;
        if (w && e + j < E) {
          o[j] += row_c[e + j];
          row_c[e + j] = 0.f;
        }
      }
      if (in && e < E) {
        if constexpr (VEC == 4)
          *reinterpret_cast<float4*>(d + t * ldd + e) = make_float4(o[0], o[1], o[2], o[3]);
        else
          d[t * ldd + e] = o[0];
      }
    }
  }
}

// Lanes a token's row is spread over and loads per lane.
struct RowMap {
  int vec, L, V;
};
RowMap row_map(int E, bool vec4) {
  RowMap m;
  m.vec = vec4 ? 4 : 1;
  const int words = (E + m.vec - 1) / m.vec;
  m.L = 1;
  while (m.L < words && m.L < 32) m.L <<= 1;
  const int v = (words + m.L - 1) / m.L;
  m.V = v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 8;
  return m;
}

// Calls fn with the kernel's template arguments as integral constants.
template <class F>
void with_map(const RowMap& m, F&& fn) {
  using std::integral_constant;
  if (m.vec == 4) {
    if (m.V == 1) fn(integral_constant<int, 4>(), integral_constant<int, 1>());
    else fn(integral_constant<int, 4>(), integral_constant<int, 2>());
  } else if (m.V == 1) {
    fn(integral_constant<int, 1>(), integral_constant<int, 1>());
  } else if (m.V == 2) {
    fn(integral_constant<int, 1>(), integral_constant<int, 2>());
  } else if (m.V == 4) {
    fn(integral_constant<int, 1>(), integral_constant<int, 4>());
  } else {
    fn(integral_constant<int, 1>(), integral_constant<int, 8>());
  }
}

int router_blocks(int64_t T, const RowMap& m, int per_warp, int most) {
  const int64_t per_block = (int64_t)kWarps * (32 / m.L) * per_warp;
  return (int)std::max<int64_t>(1, std::min<int64_t>((T + per_block - 1) / per_block, most));
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

moe_status_t check_sizes(int32_t T, int32_t E, int32_t k, int64_t ld) {
  if (E < 1 || E > 256) return fail(MOE_ERR_INVALID_ARG, "E=%d outside [1,256]", E);
  if (k < 1 || k > 8 || k > E)
    return fail(MOE_ERR_INVALID_ARG, "k=%d must be in [1, min(E,8)]", k);
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d is negative", T);
  if (ld < E) return fail(MOE_ERR_INVALID_ARG, "ld_logits must be >= E");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_router_loss_workspace(int32_t E) {
  if (E < 1 || E > 256) {
    fail(MOE_ERR_INVALID_ARG, "E=%d outside [1,256]", E);
    return 0;
  }
  return (size_t)kMaxBlocks * (E + 1) * sizeof(Partial);
}

moe_status_t moe_router_loss_fwd(const float* logits, int64_t ld_logits, const int32_t* topk_ids,
                                 const uint8_t* token_mask, int32_t T, int32_t E, int32_t k,
                                 float coef, float* loss, int32_t* counts, float* mean_prob,
                                 int32_t* n_valid, void* ws, size_t ws_bytes,
                                 moe_stream_t stream) {
  moe_status_t st = check_sizes(T, E, k, ld_logits);
  if (st != MOE_OK) return st;
  if ((T > 0 && (!logits || !topk_ids)) || !loss || !counts || !mean_prob || !n_valid || !ws)
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!a4(logits) || !a4(topk_ids) || !a4(loss) || !a4(counts) || !a4(mean_prob) || !a4(n_valid))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be 4-byte aligned");
  if (!a16(ws)) return fail(MOE_ERR_INVALID_ARG, "ws must be 16-byte aligned");
  if (ws_bytes < moe_router_loss_workspace(E))
    return fail(MOE_ERR_WORKSPACE, "ws_bytes=%zu < required %zu", ws_bytes,
                moe_router_loss_workspace(E));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RowMap m = row_map(E, E % 4 == 0 && ld_logits % 4 == 0 && a16(logits));
  const int nblk = router_blocks(T, m, 2, std::min(std::max(device_sms(), 1), kMaxBlocks));
  Partial* part = static_cast<Partial*>(ws);
  with_map(m, [&](auto vec, auto v) {
    router_loss_kernel<vec.value, v.value><<<nblk, kThreads, 0, s>>>(
        logits, ld_logits, topk_ids, token_mask, T, E, k, m.L, part);
  });
  count_launch(s, MOE_K_ROUTER_LOSS);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "router loss launch");
  e = launch_chained(router_loss_finish_kernel, 1, 1024, 0, s, (const Partial*)part, nblk, E, k,
                     coef, loss, counts, mean_prob, n_valid);
  count_launch(s, MOE_K_ROUTER_LOSS);
  if (e != cudaSuccess) return cuda_fail(e, "router loss finish launch");
  return MOE_OK;
}

moe_status_t moe_router_loss_bwd(const float* logits, int64_t ld_logits, const int32_t* topk_ids,
                                 const float* topk_probs, const float* d_probs,
                                 const uint8_t* token_mask, int32_t T, int32_t E, int32_t k,
                                 float coef, const float* d_loss, const int32_t* counts,
                                 const int32_t* n_valid, float* d_logits, int64_t ld_d,
                                 moe_stream_t stream) {
  moe_status_t st = check_sizes(T, E, k, ld_logits);
  if (st != MOE_OK) return st;
  if (ld_d < E) return fail(MOE_ERR_INVALID_ARG, "ld_d must be >= E");
  if ((topk_probs != nullptr) != (d_probs != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "topk_probs and d_probs go together");
  if (!counts || !n_valid || (T > 0 && (!logits || !topk_ids || !d_logits)))
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!a4(logits) || !a4(topk_ids) || !a4(topk_probs) || !a4(d_probs) || !a4(d_loss) ||
      !a4(counts) || !a4(n_valid) || !a4(d_logits))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be 4-byte aligned");
  if (T == 0) return MOE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RowMap m = row_map(E, E % 4 == 0 && ld_logits % 4 == 0 && ld_d % 4 == 0 && a16(logits) &&
                                  a16(d_logits));
  const int nblk = router_blocks(T, m, 1, std::max(device_sms(), 1) * 8);
  with_map(m, [&](auto vec, auto v) {
    router_grad_kernel<vec.value, v.value><<<nblk, kThreads, 0, s>>>(
        logits, ld_logits, topk_ids, topk_probs, d_probs, token_mask, T, E, k, m.L, coef, d_loss,
        counts, n_valid, d_logits, ld_d);
  });
  count_launch(s, MOE_K_ROUTER_GRAD);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "router gradient launch");
  return MOE_OK;
}

}  // extern "C"
