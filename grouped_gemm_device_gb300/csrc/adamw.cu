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
  int16_t p_bf16, g_bf16;
  int16_t wide;   // its arrays lie on boundaries of eight elements (16 bytes at least)
  int16_t unused;
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

// m, v and sqrt(v) after the step; v2 the second moment before it.
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
// The quotient within two steps: r rb + eps is 0 or between 2^-75 and 2^126.
MOE_DEVICE float update(float p, const Moments& o, float lr_decay, const Now& n, const Step& s) {
  return (p - p * lr_decay) - n.a * __fdividef(o.m, o.r * n.rb + s.eps);
}

// 8 fp32 or 16 bytes in one access; streamed data is not kept in L1.
MOE_DEVICE void load8(const void* p, float (&x)[8]) {
  asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]),
                 "=f"(x[6]), "=f"(x[7])
               : "l"(p));
}
MOE_DEVICE void store8(void* p, const float (&x)[8]) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(x[0]),
               "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
               : "memory");
}
MOE_DEVICE uint4 load4(const void* p) {
  uint4 q;
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
               : "l"(p));
  return q;
}
MOE_DEVICE uint2 load2(const void* p) {
  uint2 q;
  asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(q.x), "=r"(q.y) : "l"(p));
  return q;
}
MOE_DEVICE uint32_t byte_of(const uint2& q, int j) {  // j is a constant after unrolling
  return ((j < 4 ? q.x : q.y) >> (8 * (j & 3))) & 255u;
}

// A block of 256: lane i has elements 8 i .. 8 i + 7 (WIDE: a full block whose arrays allow whole
// vectors), or every 32nd element from i on.
template <int BITS, bool WIDE>
MOE_DEVICE void adamw_block(const Tensor& t, int64_t blk, int lane, const Now& n, const Step& s) {
  const int64_t e0 = blk * kBlock + (WIDE ? lane * 8 : lane);
  auto at = [&](int j) { return WIDE ? e0 + j : e0 + j * 32; };
  auto in = [&](int j) { return WIDE || at(j) < t.numel; };
  float* weights = t.p_bf16 ? t.master : static_cast<float*>(t.p);
  float g[8], p[8], m[8], v[8];
  uint32_t sm = 0, sv = 0;
  if constexpr (BITS == 8) {
    sm = t.m_scale[blk];
    sv = t.v_scale[blk];
  }
  if constexpr (WIDE) {
    uint4 gq;
    uint2 mc, vc;
    if (t.g_bf16) gq = load4(static_cast<const __nv_bfloat16*>(t.g) + e0);
    else load8(static_cast<const float*>(t.g) + e0, g);
    load8(weights + e0, p);
    if constexpr (BITS == 8) {
      mc = load2(static_cast<const uint8_t*>(t.m) + e0);
      vc = load2(static_cast<const uint8_t*>(t.v) + e0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = decode_m(byte_of(mc, j), sm);
        v[j] = decode_r(byte_of(vc, j), sv);
      }
    } else {
      load8(static_cast<const float*>(t.m) + e0, m);
      load8(static_cast<const float*>(t.v) + e0, v);
    }
    if (t.g_bf16) {
      const uint32_t w[4] = {gq.x, gq.y, gq.z, gq.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        g[2 * j] = bf16_lo(w[j]);
        g[2 * j + 1] = bf16_hi(w[j]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      g[j] = p[j] = m[j] = v[j] = 0.f;
      if (!in(j)) continue;
      const int64_t e = at(j);
      g[j] = t.g_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.g)[e])
                      : static_cast<const float*>(t.g)[e];
      p[j] = weights[e];
      if constexpr (BITS == 8) {
        m[j] = decode_m(static_cast<const uint8_t*>(t.m)[e], sm);
        v[j] = decode_r(static_cast<const uint8_t*>(t.v)[e], sv);
      } else {
        m[j] = static_cast<const float*>(t.m)[e];
        v[j] = static_cast<const float*>(t.v)[e];
      }
    }
  }
  const float lr_decay = n.lr * t.decay;
  uint32_t most_m = 0, most_r = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if constexpr (BITS == 8) v[j] = __fmul_rn(v[j], v[j]);
    const Moments o = advance(__fmul_rn(g[j], n.factor), m[j], v[j], s);
    p[j] = update(p[j], o, lr_decay, n, s);
    m[j] = o.m;
    v[j] = BITS == 8 ? o.r : o.v;
    if constexpr (BITS == 8) {  // elements past the end are 0
      most_m = max(most_m, __float_as_uint(fabsf(o.m)));
      most_r = max(most_r, __float_as_uint(fabsf(o.r)));
    }
  }
  if constexpr (WIDE) {
    store8(weights + e0, p);
    if (t.p_bf16)
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(t.p) + e0) =
          make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                     pack_bf16x2(p[6], p[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (in(j)) {
        weights[at(j)] = p[j];
        if (t.p_bf16) static_cast<__nv_bfloat16*>(t.p)[at(j)] = __float2bfloat16_rn(p[j]);
      }
  }
  if constexpr (BITS == 32) {
    if constexpr (WIDE) {
      store8(static_cast<float*>(t.m) + e0, m);
      store8(static_cast<float*>(t.v) + e0, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (in(j)) {
          static_cast<float*>(t.m)[at(j)] = m[j];
          static_cast<float*>(t.v)[at(j)] = v[j];
        }
    }
  } else {
    sm = block_scale(__reduce_max_sync(0xFFFFFFFFu, most_m));
    sv = block_scale(__reduce_max_sync(0xFFFFFFFFu, most_r));
    const uint32_t key = mix((uint32_t)(e0 >> 32) ^ mix((uint32_t)t.index + n.key));
    uint32_t cm[8], cv[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = mix((uint32_t)at(j) ^ key);
      cm[j] = encode(fabsf(m[j]), w & 0xFFFFu, sm, 127);
      if (m[j] < 0.f && cm[j]) cm[j] |= 128u;
      cv[j] = encode(v[j], w >> 16, sv, 255);
    }
    if constexpr (WIDE) {
      auto bytes = [](const uint32_t(&c)[8]) {
        return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                          c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
      };
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + e0) = bytes(cm);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + e0) = bytes(cv);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (in(j)) {
          static_cast<uint8_t*>(t.m)[at(j)] = (uint8_t)cm[j];
          static_cast<uint8_t*>(t.v)[at(j)] = (uint8_t)cv[j];
        }
    }
    if (lane == 0) {
      t.m_scale[blk] = (uint8_t)sm;
      t.v_scale[blk] = (uint8_t)sv;
    }
  }
}

// Four blocks an SM: 403 M elements with 32-bit states 1740 us, with three 1826, with five (registers
// for one) 1903.
template <int BITS>
__global__ void __launch_bounds__(kThreads, 4) adamw_kernel(const __grid_constant__ Batch b,
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
    const int64_t blk = c - t.first;
    if (t.wide && (blk + 1) * kBlock <= t.numel) adamw_block<BITS, true>(t, blk, lane, n, s);
    else adamw_block<BITS, false>(t, blk, lane, n, s);
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
    if (t.wide && e0 + kBlock <= t.numel) {
      const int64_t e = e0 + lane * 8;
      const uint2 mc = load2(static_cast<const uint8_t*>(t.m) + e);
      const uint2 vc = load2(static_cast<const uint8_t*>(t.v) + e);
      float m[8], v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        m[j] = decode_m(byte_of(mc, j), sm);
        v[j] = decode_r(byte_of(vc, j), sv);
      }
      *reinterpret_cast<uint4*>(out.m[i] + e) = make_uint4(
          pack_bf16x2(m[0], m[1]), pack_bf16x2(m[2], m[3]), pack_bf16x2(m[4], m[5]),
          pack_bf16x2(m[6], m[7]));
      *reinterpret_cast<uint4*>(out.v[i] + e) = make_uint4(
          pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
          pack_bf16x2(v[6], v[7]));
      continue;
    }
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
int fill_batch(Batch& b, int i, int n, const moe_adamw_tensor_t* list, int bits) {
  b.n = 0;
  b.blocks = 0;
  const int state = bits == 8 ? 8 : 32;  // bytes of eight values
  for (; i < n && b.n < kCap; ++i) {
    const moe_adamw_tensor_t& l = list[i];
    if (l.numel == 0) continue;
    const int pb = l.param_dtype == MOE_DT_BF16, gb = l.grad_dtype == MOE_DT_BF16;
    const bool wide = on(l.param, pb ? 16 : 32) && on(l.master, 32) && on(l.grad, gb ? 16 : 32) &&
                      on(l.m, state) && on(l.v, state);
    b.t[b.n++] = {l.param, l.master, l.grad, l.m, l.v, l.m_scale, l.v_scale, l.numel, b.blocks,
                  l.decay, i, (int16_t)pb, (int16_t)gb, (int16_t)wide, 0};
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
    i = fill_batch(b, i, n, tensors, state_bits);
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
  for (int i = 0; i < n;) {
    i = fill_batch(b, i, n, tensors, 8);
    if (b.n == 0) break;
    for (int j = 0; j < b.n; ++j) {
      out.m[j] = static_cast<__nv_bfloat16*>(m_out[b.t[j].index]);
      out.v[j] = static_cast<__nv_bfloat16*>(v_out[b.t[j].index]);
      b.t[j].wide = on(b.t[j].m, 8) && on(b.t[j].v, 8) && on(out.m[j], 16) && on(out.v[j], 16);
    }
    const cudaError_t e = launch_pdl(adamw_moments_kernel, adamw_blocks<adamw_moments_kernel>(b.blocks),
                                     kThreads, 0, s, 1, b, out);
    count_launch(s, MOE_K_ADAMW_MOMENTS);
    if (e != cudaSuccess) return cuda_fail(e, "AdamW moments launch");
  }
  return MOE_OK;
}

}  // extern "C"
