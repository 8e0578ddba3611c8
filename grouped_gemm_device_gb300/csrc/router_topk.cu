// Choice of experts and the gradient of its weights (moe_router_topk_fwd / moe_router_topk_bwd in
// include/moegmm.h).
//
//   s = sigmoid(l) or softmax(l);  v = s + bias;  the best groups, their best k experts;
//   w = scale s, or scale s / sum of the chosen s
//
// A warp has a token; lane i holds the VPL neighbouring experts i VPL .., so that the lowest lane
// that holds a maximum holds the lowest index, and a tree over lanes adds neighbours first.
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kWeightEps = 1e-20f;  // added to the sum that sigmoid scores are divided by

MOE_DEVICE float to_f(float v) { return v; }
MOE_DEVICE float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }

// Unsigned numbers in the order of floats, +0 and -0 the same; never 0.
MOE_DEVICE uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// The VPL logits of a lane; NaN and what lies past E read as -inf.
template <int VPL, typename LT>
MOE_DEVICE void load_logits(const LT* row, int E, int lane, float (&v)[VPL]) {
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane * VPL + j;
    v[j] = e < E ? fmaxf(to_f(row[e]), -INFINITY) : -INFINITY;
  }
}

MOE_DEVICE float sigmoid(float x) { return __frcp_rn(1.0f + expf(-x)); }

MOE_DEVICE float warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// Row sum, neighbours in pairs and then pairs of pairs.
template <int VPL>
MOE_DEVICE float pair_sum(const float (&v)[VPL]) {
  float a[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) a[j] = v[j];
#pragma unroll
  for (int w = 1; w < VPL; w <<= 1)
#pragma unroll
    for (int j = 0; j < VPL; j += 2 * w) a[j] = __fadd_rn(a[j], a[j + w]);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) a[0] = __fadd_rn(a[0], __shfl_xor_sync(kAll, a[0], o));
  return a[0];
}
// Softmax of a row in place: exp(x - max), 1 where x is the maximum, times the sum's reciprocal.
template <int VPL>
MOE_DEVICE void softmax_row(float (&v)[VPL], int E, int lane) {
  float m = v[0];
#pragma unroll
  for (int j = 1; j < VPL; ++j) m = fmaxf(m, v[j]);
  m = warp_max(m);
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const float e = v[j] == m ? 1.0f : expf(v[j] - m);
    v[j] = lane * VPL + j < E ? e : 0.f;
  }
  const float inv = __frcp_rn(pair_sum(v));
#pragma unroll
  for (int j = 0; j < VPL; ++j) v[j] = __fmul_rn(v[j], inv);
}
// Sum over lanes 0 .. 7 (and every other eight of the warp).
MOE_DEVICE float sum8(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
  return x;
}
MOE_DEVICE float max8(float x) {
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
  return x;
}

struct Choice {
  int E, k, score, n_group, topk_group, group_top, renorm;
  float scale;
};

// The largest of the warp's keys, the lowest index among equal ones; its key becomes 0.
template <int VPL>
MOE_DEVICE int take_best(uint32_t (&key)[VPL], int lane) {
  uint32_t m = key[0];
#pragma unroll
  for (int j = 1; j < VPL; ++j) m = max(m, key[j]);
  const uint32_t best = __reduce_max_sync(kAll, m);
  const int owner = __ffs(__ballot_sync(kAll, m == best)) - 1;
  int at = 0;
#pragma unroll
  for (int j = VPL - 1; j >= 0; --j)
    if (key[j] == best) at = j;
  if (lane == owner) {
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (j == at) key[j] = 0;
  }
  return owner * VPL + __shfl_sync(kAll, at, owner);
}

template <int VPL, typename LT>
__global__ void __launch_bounds__(kThreads) router_topk_kernel(
    const LT* __restrict__ logits, int64_t ld, const float* __restrict__ bias,
    const uint8_t* __restrict__ mask, int T, const Choice c, int32_t* __restrict__ ids,
    float* __restrict__ weights, int32_t* __restrict__ counts) {
  MOE_GRIDDEP_ENTRY();
  __shared__ int hist[256];
  __shared__ float by_expert[kWarps][2][256];  // choice and value; then the groups' marks
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = c.E, k = c.k;
  if (counts) {
    for (int i = threadIdx.x; i < E; i += kThreads) hist[i] = 0;
    __syncthreads();
  }
  float b[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) b[j] = bias && lane * VPL + j < E ? bias[lane * VPL + j] : 0.f;
  float(&ch)[256] = by_expert[warp][0];
  float(&va)[256] = by_expert[warp][1];
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < T; t += (int64_t)gridDim.x * kWarps) {
    if (mask && !mask[t]) {
      if (lane < k) {
        ids[t * k + lane] = -1;
        weights[t * k + lane] = 0.f;
      }
      continue;
    }
    const LT* row = logits + t * ld;
    float x[VPL], s[VPL], v[VPL];
    load_logits<VPL>(row, E, lane, x);
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = x[j];
    if (c.score == MOE_SCORE_SIGMOID) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) s[j] = sigmoid(s[j]);
    } else {
      softmax_row<VPL>(s, E, lane);
    }
    uint32_t key[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      v[j] = bias ? fmaxf(__fadd_rn(s[j], b[j]), -INFINITY) : s[j];
      key[j] = lane * VPL + j < E ? ordered(bias ? v[j] : x[j]) : 0u;
    }
    if (c.n_group > 1) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        ch[lane * VPL + j] = bias ? v[j] : x[j];
        va[lane * VPL + j] = v[j];
      }
      __syncwarp();
      const int size = E / c.n_group;
      uint32_t gkey[VPL];  // a group a place, as the experts
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const int grp = lane * VPL + j;
        gkey[j] = 0;
        if (grp < c.n_group) {
          float best = -INFINITY, next = -INFINITY;
          for (int i = grp * size; i < (grp + 1) * size; ++i) {
            const float a = c.group_top == 1 ? ch[i] : va[i];
            next = fmaxf(next, fminf(a, best));
            best = fmaxf(best, a);
          }
          gkey[j] = ordered(c.group_top == 1 ? best : fmaxf(__fadd_rn(best, next), -INFINITY));
        }
      }
      __syncwarp();
      for (int i = lane; i < c.n_group; i += 32) ch[i] = 0.f;
      __syncwarp();
      for (int i = 0; i < c.topk_group; ++i) {
        const int grp = take_best<VPL>(gkey, lane);
        if (lane == 0) ch[grp] = 1.f;
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (lane * VPL + j < E && ch[(lane * VPL + j) / size] == 0.f) key[j] = 0;
      __syncwarp();
    }
    int mine = 0;  // lane j < k: the j-th expert
    for (int j = 0; j < k; ++j) {
      const int e = take_best<VPL>(key, lane);
      if (lane == j) mine = e;
    }
    const bool live = lane < k;
    const float l = live ? fmaxf(to_f(row[mine]), -INFINITY) : -INFINITY;
    float w;
    if (c.renorm && c.score == MOE_SCORE_SOFTMAX) {
      const float m = max8(l);
      w = live ? (l == m ? 1.0f : expf(l - m)) : 0.f;
      w = w / sum8(w);
    } else {
      // the score of expert `mine`
      w = 0.f;
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float other = __shfl_sync(kAll, s[j], mine / VPL);
        if (mine % VPL == j) w = other;
      }
      if (!live) w = 0.f;
      if (c.renorm) w = w / (sum8(w) + kWeightEps);
    }
    if (live) {
      ids[t * k + lane] = mine;
      weights[t * k + lane] = w * c.scale;
      if (counts) atomicAdd(&hist[mine], 1);
    }
  }
  if (!counts) return;
  __syncthreads();
  for (int i = threadIdx.x; i < E; i += kThreads) {
    if (gridDim.x == 1) counts[i] = hist[i];
    else if (hist[i]) atomicAdd(&counts[i], hist[i]);
  }
}

// A warp has a token: its lanes 0 .. k - 1 the slots' parts, each lane then the VPL experts it owns.
template <int VPL, typename LT>
__global__ void __launch_bounds__(kThreads) router_topk_grad_kernel(
    const LT* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, int T, int E, int k, int score, int renorm, float scale,
    const float* add_to, int64_t ld_add, float* d, int64_t ldd) {
  MOE_GRIDDEP_ENTRY();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool whole = score == MOE_SCORE_SOFTMAX && !renorm;
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < T; t += (int64_t)gridDim.x * kWarps) {
    const LT* row = logits + t * ld;
    int e = -1;
    float u = 0.f, l = -INFINITY;
    if (lane < k) {
      e = ids[t * k + lane];
      if (e < 0 || e >= E) e = -1;
      if (e >= 0) {
        u = dw[t * k + lane] * scale;
        l = fmaxf(to_f(row[e]), -INFINITY);
      }
    }
    if (score == MOE_SCORE_SIGMOID) {
      const float q = expf(-fabsf(l)), r = 1.0f / (1.0f + q);
      const float s = l >= 0.f ? r : q * r;
      if (renorm) {
        const float sc = e >= 0 ? s : 0.f, total = sum8(sc) + kWeightEps;
        u = (u - sum8(u * sc) / total) / total;
      }
      u *= q * r * r;  // s (1 - s)
    } else if (renorm) {
      const float m = max8(l);
      float w = e >= 0 ? (l == m ? 1.0f : expf(l - m)) : 0.f;
      w = w / fmaxf(sum8(w), 1.0f);  // at least the maximum's 1, but for a token without slots
      u = w * (u - sum8(w * u));
    }
    if (e < 0) u = 0.f;
    float o[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) o[j] = 0.f;
    for (int i = 0; i < k; ++i) {
      const int at = __shfl_sync(kAll, e, i) - lane * VPL;
      const float y = __shfl_sync(kAll, u, i);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (at == j) o[j] += y;
    }
    if (whole) {
      float p[VPL], a = 0.f;
      load_logits<VPL>(row, E, lane, p);
      softmax_row<VPL>(p, E, lane);
#pragma unroll
      for (int j = 0; j < VPL; ++j) a += p[j] * o[j];
#pragma unroll
      for (int q = 16; q > 0; q >>= 1) a += __shfl_xor_sync(kAll, a, q);
#pragma unroll
      for (int j = 0; j < VPL; ++j) o[j] = p[j] * (o[j] - a);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int i = lane * VPL + j;
      if (i < E) d[t * ldd + i] = add_to ? add_to[t * ld_add + i] + o[j] : o[j];
    }
  }
}

template <int N>
using I = std::integral_constant<int, N>;
// Calls fn with the experts a lane and a value of the logits' type.
template <class F>
void with_shape(int E, int32_t dtype, F&& fn) {
  auto typed = [&](auto vpl) {
    if (dtype == MOE_DT_FP32) fn(vpl, float());
    else fn(vpl, __nv_bfloat16());
  };
  if (E <= 32) typed(I<1>());
  else if (E <= 64) typed(I<2>());
  else if (E <= 128) typed(I<4>());
  else typed(I<8>());
}

int topk_blocks(int64_t T) {
  return (int)std::max<int64_t>(
      1, std::min<int64_t>((T + kWarps - 1) / kWarps, (int64_t)std::max(device_sms(), 1) * 8));
}

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

moe_status_t check_shape(int32_t T, int32_t E, int32_t k, int64_t ld, int32_t dtype,
                         int32_t score) {
  if (E < 1 || E > 256) return fail(MOE_ERR_INVALID_ARG, "E=%d outside [1,256]", E);
  if (k < 1 || k > 8 || k > E)
    return fail(MOE_ERR_INVALID_ARG, "k=%d must be in [1, min(E,8)]", k);
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d is negative", T);
  if (ld < E) return fail(MOE_ERR_INVALID_ARG, "ld_logits must be >= E");
  if (dtype != MOE_DT_BF16 && dtype != MOE_DT_FP32)
    return fail(MOE_ERR_INVALID_ARG, "unknown logits_dtype %d", dtype);
  if (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID)
    return fail(MOE_ERR_INVALID_ARG, "unknown score %d", score);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_router_topk_fwd(const void* logits, int64_t ld_logits, int32_t logits_dtype,
                                 const float* bias, const uint8_t* token_mask, int32_t T,
                                 int32_t E, int32_t k, int32_t score, int32_t n_group,
                                 int32_t topk_group, int32_t group_top, int32_t renorm,
                                 float scale, int32_t* topk_ids, float* topk_weights,
                                 int32_t* counts, moe_stream_t stream) {
  moe_status_t st = check_shape(T, E, k, ld_logits, logits_dtype, score);
  if (st != MOE_OK) return st;
  if (n_group < 1 || E % n_group)
    return fail(MOE_ERR_INVALID_ARG, "n_group=%d must divide E=%d", n_group, E);
  if (topk_group < 1 || topk_group > n_group || topk_group * (E / n_group) < k)
    return fail(MOE_ERR_INVALID_ARG, "topk_group=%d outside [1, n_group], or too few experts for k",
                topk_group);
  if (group_top != 1 && group_top != 2)
    return fail(MOE_ERR_INVALID_ARG, "group_top=%d must be 1 or 2", group_top);
  if (group_top == 2 && E / n_group < 2)
    return fail(MOE_ERR_INVALID_ARG, "group_top 2 needs two experts a group");
  if (T > 0 && (!logits || !topk_ids || !topk_weights))
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!on(logits, logits_dtype == MOE_DT_FP32 ? 4 : 2) || !on(bias, 4) || !on(topk_ids, 4) ||
      !on(topk_weights, 4) || !on(counts, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int grid = topk_blocks(T);
  cudaError_t e = cudaSuccess;
  if (T == 0 || grid > 1) {  // a single block writes the counts, several add to them
    if (counts) e = cudaMemsetAsync(counts, 0, sizeof(int32_t) * E, s);
    if (e != cudaSuccess) return cuda_fail(e, "memset counts");
    if (T == 0) return MOE_OK;
  }
  const Choice c = {E, k, score, n_group, topk_group, group_top, renorm != 0, scale};
  with_shape(E, logits_dtype, [&](auto vpl, auto lt) {
    using LT = decltype(lt);
    e = launch_pdl(router_topk_kernel<vpl.value, LT>, grid, kThreads, 0, s, 1,
                   static_cast<const LT*>(logits), ld_logits, bias, token_mask, T, c, topk_ids,
                   topk_weights, counts);
  });
  count_launch(s, MOE_K_ROUTER_TOPK);
  if (e != cudaSuccess) return cuda_fail(e, "router top-k launch");
  return MOE_OK;
}

moe_status_t moe_router_topk_bwd(const void* logits, int64_t ld_logits, int32_t logits_dtype,
                                 const int32_t* topk_ids, const float* d_weights, int32_t T,
                                 int32_t E, int32_t k, int32_t score, int32_t renorm, float scale,
                                 const float* add_to, int64_t ld_add, float* d_logits,
                                 int64_t ld_d, moe_stream_t stream) {
  moe_status_t st = check_shape(T, E, k, ld_logits, logits_dtype, score);
  if (st != MOE_OK) return st;
  if (ld_d < E || (add_to && ld_add < E))
    return fail(MOE_ERR_INVALID_ARG, "row strides must be >= E");
  if (T > 0 && (!logits || !topk_ids || !d_weights || !d_logits))
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  if (add_to == d_logits && add_to && ld_add != ld_d)
    return fail(MOE_ERR_INVALID_ARG, "add_to is d_logits, with another row stride");
  if (!on(logits, logits_dtype == MOE_DT_FP32 ? 4 : 2) || !on(topk_ids, 4) || !on(d_weights, 4) ||
      !on(add_to, 4) || !on(d_logits, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (T == 0) return MOE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  with_shape(E, logits_dtype, [&](auto vpl, auto lt) {
    using LT = decltype(lt);
    e = launch_pdl(router_topk_grad_kernel<vpl.value, LT>, topk_blocks(T), kThreads, 0, s, 1,
                   static_cast<const LT*>(logits), ld_logits, topk_ids, d_weights, T, E, k, score,
                   renorm != 0, scale, add_to, ld_add, d_logits, ld_d);
  });
  count_launch(s, MOE_K_ROUTER_TOPK_GRAD);
  if (e != cudaSuccess) return cuda_fail(e, "router top-k gradient launch");
  return MOE_OK;
}

}  // extern "C"
