// AdamW over a list of tensors, states in 32 or 8 bits (moe_adamw_step and moe_adamw_moments in
// include/moegmm.h, which defines the step, the 8-bit format and its rounding).
//
// Bound by HBM: an element's weight, gradient and states are read once and written once. A warp takes
// 256 elements at a time, the block that shares a scale in an 8-bit state. The step's scalars (bias
// corrections, clip factor, learning rate) come from device memory and are formed once a block, so
// that a captured step replays as the next one. The steps are counted by the last block to finish.
// m, v and r = sqrt(v) are formed by single rounded fp32 operations (no contraction): which code a
// value gets does not depend on how the compiler joins them.
#include <cmath>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;       // elements that share a scale
constexpr int kCap = 40;          // tensors a launch: they travel as kernel parameters
constexpr float kClipEps = 1e-6f;
constexpr uint32_t kNanScale = 255, kLowScale = 32;

struct Tensor {
  void* p;
  float* master;
  const void* g;
  void *m, *v;
  uint8_t *m_scale, *v_scale;
  int64_t numel;
  int64_t first;  // its first block of 256 among the launch's
  float decay;
  int32_t index;  // in the caller's list
  int16_t p_bf16, g_bf16, vec, unused;
};
struct Batch {
  Tensor t[kCap];
  int n;
  int64_t blocks;
};
struct Step {
  float lr, b1, c1, b2, c2, eps, max_norm;  // c = 1 - b
  double log_b1, log_b2;
  const float *lr_dev, *norm;
  uint32_t seed_lo, seed_hi;
  unsigned long long* counters;
  int last;  // the step's last launch counts it
};

MOE_DEVICE int find_tensor(const Batch& b, int64_t block) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.t[mid].first <= block) lo = mid; else hi = mid;
  }
  return lo;
}

// 32-bit hash; a change of any input bit changes each output bit in half of the cases (to 0.1%,
// measured over 2^18 words).
MOE_DEVICE uint32_t mix(uint32_t x) {
  x ^= x >> 16;
  x *= 0xf75341d5u;
  x ^= x >> 15;
  x *= 0x99d5d0a1u;
  return x ^ (x >> 16);
}

// The value of a code: the top 12 bits of an fp32 number, counted from `base`.
MOE_DEVICE int code_base(uint32_t scale, int top) { return (int)scale * 8 + 7 - top; }
MOE_DEVICE float decode(uint32_t mag, int base, uint32_t scale) {
  if (scale == kNanScale) return __uint_as_float(0x7FC00000u);
  return mag == 0 ? 0.f : __uint_as_float((uint32_t)(base + (int)mag) << 20);
}
MOE_DEVICE float decode_m(uint32_t code, uint32_t scale) {
  const float x = decode(code & 127u, code_base(scale, 127), scale);
  return code & 128u ? -x : x;
}
MOE_DEVICE float decode_r(uint32_t code, uint32_t scale) {
  return decode(code, code_base(scale, 255), scale);
}
// The scale of a block whose largest magnitude has these bits, rounded up to a code.
MOE_DEVICE uint32_t block_scale(uint32_t most) {
  const uint32_t s = (most + 0xFFFFFu) >> 23;
  return s < kLowScale ? kLowScale : s > kNanScale ? kNanScale : s;
}
// The code of magnitude x >= 0, one of its two neighbours by 16 random bits.
MOE_DEVICE uint32_t encode(float x, uint32_t u, uint32_t scale, int top) {
  if (scale == kNanScale) return 0u;
  const int base = code_base(scale, top);
  const float least = __uint_as_float((uint32_t)(base + 1) << 20);
  if (x < least) return (float)u * (least * 0x1p-16f) < x ? 1u : 0u;
  return ((__float_as_uint(x) + (u << 4)) >> 20) - (uint32_t)base;
}

// Scalars of a step, the same in every thread of a block.
struct Now {
  float a, rb, lr, factor;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t key;             // of the step's random words
  unsigned long long t;
  int skip;
};
MOE_DEVICE Now step_now(const Step& s) {
  Now n;
  n.t = s.counters[0] + 1;
  n.lr = s.lr_dev ? *s.lr_dev : s.lr;
  // 1 - b^t = -expm1(t log b), the exponent in fp64
  n.a = n.lr / -expm1f((float)((double)n.t * s.log_b1));
  n.rb = 1.0f / sqrtf(-expm1f((float)((double)n.t * s.log_b2)));
  n.factor = 1.0f;
  n.skip = 0;
  if (s.norm) {
    const float norm = *s.norm;
    n.skip = !(norm < INFINITY);
    n.factor = fminf(s.max_norm / (norm + kClipEps), 1.0f);
  }
  n.key = mix((uint32_t)n.t ^ mix(s.seed_lo ^ mix(s.seed_hi)));
  return n;
}

// m, v and the weight after the step; v2 the second moment before it.
struct Moments {
  float m, v, r;
};
MOE_DEVICE Moments advance(float g, float m, float v2, const Step& s) {
  Moments o;
  o.m = __fadd_rn(__fmul_rn(m, s.b1), __fmul_rn(g, s.c1));
  o.v = __fadd_rn(__fmul_rn(v2, s.b2), __fmul_rn(__fmul_rn(g, s.c2), g));
  o.r = __fsqrt_rn(o.v);
  return o;
}
MOE_DEVICE float update(float p, const Moments& o, float lr_decay, const Now& n, const Step& s) {
  return (p - p * lr_decay) - n.a * (o.m / (o.r * n.rb + s.eps));
}

template <int BITS>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Batch b,
                                                         const __grid_constant__ Step s) {
  MOE_GRIDDEP_ENTRY();
  __shared__ Now sn;
  if (threadIdx.x == 0) sn = step_now(s);
  __syncthreads();
  const Now n = sn;
  if (n.skip) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t c = (int64_t)blockIdx.x * kWarps + warp; c < b.blocks;
       c += (int64_t)gridDim.x * kWarps) {
    const Tensor& t = b.t[find_tensor(b, c)];
    const int64_t blk = c - t.first, e0 = blk * kBlock;
    const float lr_decay = n.lr * t.decay;
    const uint32_t key = mix((uint32_t)(e0 >> 32) ^ mix((uint32_t)t.index + n.key));
    uint32_t sm = 0, sv = 0;
    if constexpr (BITS == 8) {
      sm = t.m_scale[blk];
      sv = t.v_scale[blk];
    }
    Moments o[8];
    uint32_t most_m = 0, most_r = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = e0 + j * 32 + lane;
      o[j] = {0.f, 0.f, 0.f};
      if (e >= t.numel) continue;
      float g = t.g_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.g)[e])
                         : static_cast<const float*>(t.g)[e];
      g = __fmul_rn(g, n.factor);
      float m, v;
      if constexpr (BITS == 8) {
        m = decode_m(static_cast<const uint8_t*>(t.m)[e], sm);
        const float r = decode_r(static_cast<const uint8_t*>(t.v)[e], sv);
        v = __fmul_rn(r, r);
      } else {
        m = static_cast<const float*>(t.m)[e];
        v = static_cast<const float*>(t.v)[e];
      }
      o[j] = advance(g, m, v, s);
      float* pm = t.p_bf16 ? t.master : static_cast<float*>(t.p);
      const float p = update(pm[e], o[j], lr_decay, n, s);
      pm[e] = p;
      if (t.p_bf16) static_cast<__nv_bfloat16*>(t.p)[e] = __float2bfloat16_rn(p);
      if constexpr (BITS == 8) {
        most_m = max(most_m, __float_as_uint(fabsf(o[j].m)));
        most_r = max(most_r, __float_as_uint(fabsf(o[j].r)));
      } else {
        static_cast<float*>(t.m)[e] = o[j].m;
        static_cast<float*>(t.v)[e] = o[j].v;
      }
    }
    if constexpr (BITS == 8) {
      sm = block_scale(__reduce_max_sync(0xFFFFFFFFu, most_m));
      sv = block_scale(__reduce_max_sync(0xFFFFFFFFu, most_r));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t e = e0 + j * 32 + lane;
        if (e >= t.numel) continue;
        const uint32_t w = mix((uint32_t)e ^ key);
        const uint32_t cm = encode(fabsf(o[j].m), w & 0xFFFFu, sm, 127);
        static_cast<uint8_t*>(t.m)[e] = (uint8_t)(cm | (cm && o[j].m < 0.f ? 128u : 0u));
        static_cast<uint8_t*>(t.v)[e] = (uint8_t)encode(o[j].r, w >> 16, sv, 255);
      }
      if (lane == 0) {
        t.m_scale[blk] = (uint8_t)sm;
        t.v_scale[blk] = (uint8_t)sv;
      }
    }
  }
  if (!s.last) return;
  if (threadIdx.x == 0) {  // this block's read of the count lies before its ticket
    __threadfence();
    if (atomicAdd(&s.counters[1], 1ull) == gridDim.x - 1) {
      s.counters[1] = 0;
      s.counters[0] = n.t;
    }
  }
}

struct MomentsOut {
  __nv_bfloat16 *m[kCap], *v[kCap];
};
__global__ void __launch_bounds__(kThreads) adamw_moments_kernel(const __grid_constant__ Batch b,
                                                                 const __grid_constant__ MomentsOut out) {
  MOE_GRIDDEP_ENTRY();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t c = (int64_t)blockIdx.x * kWarps + warp; c < b.blocks;
       c += (int64_t)gridDim.x * kWarps) {
    const int i = find_tensor(b, c);
    const Tensor& t = b.t[i];
    const int64_t blk = c - t.first, e0 = blk * kBlock;
    const uint32_t sm = t.m_scale[blk], sv = t.v_scale[blk];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = e0 + j * 32 + lane;
      if (e >= t.numel) continue;
      out.m[i][e] = __float2bfloat16_rn(decode_m(static_cast<const uint8_t*>(t.m)[e], sm));
      out.v[i][e] = __float2bfloat16_rn(decode_r(static_cast<const uint8_t*>(t.v)[e], sv));
    }
  }
}

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Tensors [i, ..) of the list that hold elements, up to kCap; returns the next index.
int fill_batch(Batch& b, int i, int n, const moe_adamw_tensor_t* list, int* from) {
  b.n = 0;
  b.blocks = 0;
  for (; i < n && b.n < kCap; ++i) {
    const moe_adamw_tensor_t& l = list[i];
    if (l.numel == 0) continue;
    if (from) from[b.n] = i;
    Tensor& t = b.t[b.n++];
    t = {l.param, l.master, l.grad, l.m, l.v, l.m_scale, l.v_scale, l.numel, b.blocks, l.decay, i,
         l.param_dtype == MOE_DT_BF16, l.grad_dtype == MOE_DT_BF16, 0, 0};
    b.blocks += (l.numel + kBlock - 1) / kBlock;
  }
  return i;
}

template <auto Kernel>
int adamw_blocks(int64_t blocks) {
  static DeviceCache cache;
  const int per_sm = std::max(1, cache.get(current_device(), [] {
    return blocks_per_sm(reinterpret_cast<const void*>(Kernel), kThreads, 0);
  }));
  const int64_t fit = (int64_t)std::max(device_sms(), 1) * per_sm;
  return (int)std::max<int64_t>(1, std::min((blocks + kWarps - 1) / kWarps, fit));
}

moe_status_t check_list(int32_t n, const moe_adamw_tensor_t* list, int bits, bool states_only) {
  if (n < 0 || n > 65536) return fail(MOE_ERR_INVALID_ARG, "n=%d outside [0, 65536]", n);
  if (n > 0 && !list) return fail(MOE_ERR_INVALID_ARG, "NULL host array");
  for (int i = 0; i < n; ++i) {
    const moe_adamw_tensor_t& l = list[i];
    if (l.numel < 0) return fail(MOE_ERR_INVALID_ARG, "tensor %d: negative size", i);
    if (l.numel == 0) continue;
    if (!l.m || !l.v || (bits == 8 && (!l.m_scale || !l.v_scale)))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: NULL state", i);
    if (bits == 32 && (!on(l.m, 4) || !on(l.v, 4)))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: not aligned to its elements", i);
    if (states_only) continue;
    for (int32_t d : {l.param_dtype, l.grad_dtype})
      if (d != MOE_DT_BF16 && d != MOE_DT_FP32)
        return fail(MOE_ERR_INVALID_ARG, "tensor %d: unknown dtype %d", i, d);
    if (!l.param || !l.grad) return fail(MOE_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
    if ((l.param_dtype == MOE_DT_BF16) != (l.master != nullptr))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: bf16 weights have an fp32 master, fp32 none", i);
    if (!on(l.param, l.param_dtype == MOE_DT_BF16 ? 2 : 4) || !on(l.master, 4) ||
        !on(l.grad, l.grad_dtype == MOE_DT_BF16 ? 2 : 4))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: not aligned to its elements", i);
    if (!(l.decay >= 0.f && l.decay < INFINITY))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: decay must be finite and >= 0", i);
  }
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_adamw_step(int32_t n, const moe_adamw_tensor_t* tensors, int32_t state_bits,
                            double lr, const float* lr_device, double beta1, double beta2,
                            double eps, const float* grad_norm, float max_norm, uint64_t seed,
                            int64_t* counters, moe_stream_t stream) {
  if (state_bits != 32 && state_bits != 8)
    return fail(MOE_ERR_INVALID_ARG, "state_bits=%d must be 32 or 8", state_bits);
  moe_status_t st = check_list(n, tensors, state_bits, false);
  if (st != MOE_OK) return st;
  if (!(lr >= 0 && lr < 3e38) || !(eps >= 0 && eps < 3e38))
    return fail(MOE_ERR_INVALID_ARG, "lr and eps must be finite and >= 0");
  if (!(beta1 >= 0 && beta1 < 1) || !(beta2 >= 0 && beta2 < 1))
    return fail(MOE_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!(max_norm > 0.f)) return fail(MOE_ERR_INVALID_ARG, "max_norm must be > 0");
  if (!counters || !on(counters, 8))
    return fail(MOE_ERR_INVALID_ARG, "counters must be non-NULL and 8-byte aligned");
  if (!on(lr_device, 4) || !on(grad_norm, 4))
    return fail(MOE_ERR_INVALID_ARG, "lr_device and grad_norm must be 4-byte aligned");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Step step = {(float)lr, (float)beta1, (float)(1 - beta1), (float)beta2, (float)(1 - beta2),
               (float)eps, max_norm, std::log(beta1), std::log(beta2), lr_device, grad_norm,
               (uint32_t)seed, (uint32_t)(seed >> 32),
               reinterpret_cast<unsigned long long*>(counters), 0};
  auto kernel = state_bits == 8 ? adamw_kernel<8> : adamw_kernel<32>;
  Batch b;
  int i = 0;
  do {
    i = fill_batch(b, i, n, tensors, nullptr);
    int left = i;
    while (left < n && tensors[left].numel == 0) ++left;
    step.last = left == n;
    const int grid = state_bits == 8 ? adamw_blocks<adamw_kernel<8>>(b.blocks)
                                     : adamw_blocks<adamw_kernel<32>>(b.blocks);
    const cudaError_t e = launch_pdl(kernel, grid, kThreads, 0, s, 1, b, step);
    count_launch(s, MOE_K_ADAMW);
    if (e != cudaSuccess) return cuda_fail(e, "AdamW launch");
    i = left;
  } while (i < n);
  return MOE_OK;
}

moe_status_t moe_adamw_moments(int32_t n, const moe_adamw_tensor_t* tensors, void* const* m_out,
                               void* const* v_out, moe_stream_t stream) {
  moe_status_t st = check_list(n, tensors, 8, true);
  if (st != MOE_OK) return st;
  if (n > 0 && (!m_out || !v_out)) return fail(MOE_ERR_INVALID_ARG, "NULL host array");
  for (int i = 0; i < n; ++i)
    if (tensors[i].numel > 0 && (!m_out[i] || !v_out[i] || !on(m_out[i], 2) || !on(v_out[i], 2)))
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: output NULL or not aligned", i);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Batch b;
  MomentsOut out;
  int from[kCap];
  for (int i = 0; i < n;) {
    i = fill_batch(b, i, n, tensors, from);
    if (b.n == 0) break;
    for (int j = 0; j < b.n; ++j) {
      out.m[j] = static_cast<__nv_bfloat16*>(m_out[from[j]]);
      out.v[j] = static_cast<__nv_bfloat16*>(v_out[from[j]]);
    }
    const cudaError_t e = launch_pdl(adamw_moments_kernel, adamw_blocks<adamw_moments_kernel>(b.blocks),
                                     kThreads, 0, s, 1, b, out);
    count_launch(s, MOE_K_ADAMW_MOMENTS);
    if (e != cudaSuccess) return cuda_fail(e, "AdamW moments launch");
  }
  return MOE_OK;
}

}  // extern "C"
