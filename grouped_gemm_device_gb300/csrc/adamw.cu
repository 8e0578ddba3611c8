// AdamW over a list of tensors, states in 32 or 8 bits (moe_adamw_step and moe_adamw_moments in
// include/moegmm.h, which defines the step, the 8-bit format and its rounding).
//
// Bound by HBM with 32-bit states: an element's weight, gradient and states are read once and
// written once, 28 bytes (bf16 weights with masters). 403 M elements 1600 us, 7.0 TB/s, 105% of
// the measured copy. 8-bit states move 16 bytes an element and are bound by instructions (some 75
// an element: decoding, the step, a hash, rounding): 101 M elements about 300 us, 5.4 TB/s; their
// moments read back, 6 bytes an element, about 95 us. 12 tensors of 60,001 fp32 together: 4.5 us,
// the host's. Where whole vectors cannot be used, element by element: 101 M fp32 weights off their
// boundaries 440 us with 32-bit states (floor 422), 974 to 996 with 8-bit ones. 400 equal tensors of
// 101 M take ten launches, 458 us against 407 in one. A block of threads takes 2048 elements of one tensor at a time, a warp of it the 256
// that share a scale in an 8-bit state. The step's scalars (bias corrections, clip factor,
// learning rate) come from device memory and are formed once a block, so that a captured step
// replays as the next one. The steps are counted by the last block to finish. m, v and r = sqrt(v)
// are formed by single rounded fp32 operations (no contraction): which code a value gets does not
// depend on the path.
#include <cmath>

#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 256;       // elements that share a scale
constexpr int kChunk = kWarps * kBlock;
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
  int64_t first;  // its first chunk among the launch's
  float decay;
  int32_t index;  // in the caller's list
  int16_t p_bf16, g_bf16;
  int16_t wide;   // its arrays lie on boundaries of eight elements (16 bytes at least)
  int16_t unused;
};
struct Batch {
  Tensor t[kCap];
  int n;
  int64_t chunks;
};
struct Step {
  float lr, b1, c1, b2, c2, eps, max_norm;  // c = 1 - b
  double log_b1, log_b2;
  const float *lr_dev, *norm;
  uint32_t seed_key;  // mix(seed_lo ^ mix(seed_hi))
  unsigned long long* counters;
  int last;  // the step's last launch counts it
};

MOE_DEVICE int find_tensor(const Batch& b, int64_t chunk) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.t[mid].first <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// 32-bit hash; a change of any input bit changes each output bit in half of the cases, measured over
// 2^24 random words: to 0.5% at worst (input bit 31, output bit 19), to 0.03% on average over the
// pairs of bits.
__host__ MOE_DEVICE uint32_t mix(uint32_t x) {
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

// Scalars of a step, the same in every thread of a block: three warps form a part each, so that a
// block that starts waits for the longest of them alone.
struct Now {
  float a, rb, lr, factor;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  uint32_t key;             // of the step's random words
  int skip;
  unsigned long long t;
};
MOE_DEVICE void step_now(const Step& s, Now& n) {
  if (threadIdx.x == 0) {
    n.lr = s.lr_dev ? *s.lr_dev : s.lr;
    n.t = s.counters[0] + 1;
    // 1 - b^t = -expm1(t log b), the exponent in fp64
    n.a = n.lr / -expm1f((float)((double)n.t * s.log_b1));
  } else if (threadIdx.x == 32) {
    n.rb = 1.0f / sqrtf(-expm1f((float)((double)(s.counters[0] + 1) * s.log_b2)));
  } else if (threadIdx.x == 64) {
    const float norm = s.norm ? *s.norm : 0.f;
    const uint32_t t = (uint32_t)(s.counters[0] + 1);
    n.skip = !(norm < INFINITY);
    n.factor = s.norm ? fminf(s.max_norm / (norm + kClipEps), 1.0f) : 1.0f;
    n.key = mix(t ^ s.seed_key);
  }
}

// What the low bits of element e are mixed with (the same for a chunk).
MOE_DEVICE uint32_t word_key(const Tensor& t, int64_t e, const Now& n) {
  return mix((uint32_t)(e >> 32) ^ mix((uint32_t)t.index + n.key));
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
// r rb + eps is 0 (with m / 0, as the formula has it) or between 2^-126 and 2^126, where the quotient is
// within two steps; FAR: any number, and a rounded quotient.
template <bool FAR>
MOE_DEVICE float update(float p, const Moments& o, float lr_decay, const Now& n, const Step& s) {
  const float d = o.r * n.rb + s.eps;
  return (p - p * lr_decay) - n.a * (FAR ? __fdiv_rn(o.m, d) : __fdividef(o.m, d));
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
// A lane's eight codes as pairs of bf16 numbers, which hold the four significant bits of a value: a
// code's magnitude, shifted to the fourth bit and added to the scale's base, is one.
template <bool SIGNED>
MOE_DEVICE void decode8(const uint2& q, uint32_t scale, uint32_t (&w)[4]) {
  if (scale == kNanScale) {  // the same for the whole warp
#pragma unroll
    for (uint32_t& x : w) x = 0x7FC07FC0u;
    return;
  }
  const uint32_t base = (uint32_t)code_base(scale, SIGNED ? 127 : 255) * 0x00100010u;
  uint32_t none = 0;  // marks of zeros
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = h ? q.y : q.x, mag = SIGNED ? c & 0x7F7F7F7Fu : c;
    const uint32_t lo = (c & 0x0F0F0F0Fu) << 4, hi = (mag >> 4) & 0x0F0F0F0Fu;
    const uint32_t top = SIGNED ? hi | (c & 0x80808080u) : hi;
    w[2 * h] = __byte_perm(lo, top, 0x5140) + base;
    w[2 * h + 1] = __byte_perm(lo, top, 0x7362) + base;
    none |= (mag - 0x01010101u) & ~mag & 0x80808080u;
  }
  if (none) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t c = (j < 4 ? q.x : q.y) >> (8 * (j & 3));
      if ((c & (SIGNED ? 127u : 255u)) == 0) w[j >> 1] &= j & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    }
  }
}
// The larger magnitude; a NaN stays one.
MOE_DEVICE float most_of(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(fabsf(b)));
  return m;
}
MOE_DEVICE float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Within two steps of the root (a relative 2^-23), 0 for subnormal x.
MOE_DEVICE float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
MOE_DEVICE uint32_t max_all(float x) { return __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)); }

// Writes the codes of a lane's eight m and r = sqrt(v), of elements e .. e + 7 (low 32 bits), and
// returns the block's scales. A code is the top of the value's bits plus the random ones, less the
// scale's base; with all of them shifted left by four it is a word's top byte, which drops the
// sign and what lies above a code. The root is taken approximately first (2 instructions against
// some 12): its code is the rounded one's unless two steps of r would change it, which few values
// in 10^5 need; those, and values below the least one, go a way of their own.
MOE_DEVICE uint2 hold8(const float (&m)[8], const float (&v)[8], float most_m, float most_r,
                       uint32_t e, uint32_t key, uint2* to_m, uint2* to_r) {
  const uint32_t top_m = max_all(most_m);
  uint32_t top_r = max_all(most_r);
  // near the next scale, or roots that the approximation takes for 0
  if (((top_r + 0xFFFFFu + 2) & 0x7FFFFFu) <= 4 || top_r < 0x20800000u) {  // 2^-62
    most_r = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) most_r = most_of(most_r, __fsqrt_rn(v[j]));
    top_r = max_all(most_r);
  }
  const uint32_t sm = block_scale(top_m), sr = block_scale(top_r);
  if ((top_m | top_r) == 0 || (sm & sr) == kNanScale) {
    *to_m = *to_r = make_uint2(0u, 0u);
    return make_uint2(sm, sr);
  }
  const uint32_t base_m = (uint32_t)code_base(sm, 127), base_r = (uint32_t)code_base(sr, 255);
  uint32_t ym[8], yr[8], close = ~0u;
  float low_m = INFINITY, low_r = INFINITY;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t w = mix((e + j) ^ key);
    const float r = sqrt_approx(v[j]);
    ym[j] = (__float_as_uint(m[j]) << 4) - (base_m << 24) + __byte_perm(w, 0u, 0x4104);
    yr[j] = (__float_as_uint(r) << 4) - (base_r << 24) + __byte_perm(w, 0u, 0x4324);
    close = min(close, (yr[j] << 8) + (32u << 8));
    low_m = fminf(low_m, fabsf(m[j]));
    low_r = fminf(low_r, r);
  }
  uint32_t cm[2], cr[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    auto tops = [h](const uint32_t (&y)[8]) {
      return __byte_perm(__byte_perm(y[4 * h], y[4 * h + 1], 0x0073),
                         __byte_perm(y[4 * h + 2], y[4 * h + 3], 0x0073), 0x5410);
    };
    uint32_t bits[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) bits[j] = __float_as_uint(m[j]);
    cm[h] = tops(ym) | (tops(bits) & 0x80808080u);
    cr[h] = tops(yr);
  }
  if (low_m < __uint_as_float((base_m + 1) << 20) || low_r < __uint_as_float((base_r + 2) << 20) ||
      close <= 64u << 8 || sm == kNanScale || sr == kNanScale) {
    cm[0] = cm[1] = cr[0] = cr[1] = 0u;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t w = mix((e + j) ^ key);
      uint32_t k = encode(fabsf(m[j]), w & 0xFFFFu, sm, 127);
      if (k && m[j] < 0.f) k |= 128u;
      cm[j >> 2] |= k << (8 * (j & 3));
      cr[j >> 2] |= encode(__fsqrt_rn(v[j]), w >> 16, sr, 255) << (8 * (j & 3));
    }
  }
  *to_m = make_uint2(cm[0], cm[1]);
  *to_r = make_uint2(cr[0], cr[1]);
  return make_uint2(sm, sr);
}

// 8-bit states: a block's next chunk is on its way to shared memory (cp.async, each thread its own
// bytes, so that no barrier is spent) while it works on this one: the work on 64 to 80 bytes a
// thread is long, and registers for more warps are not there. A slot holds sixteen bytes of each
// thread, four times (the gradients take one or two), then the codes' eights.
constexpr int kSlotBytes = 80 * kThreads;
constexpr int kRingBytes = 2 * kSlotBytes;
MOE_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEVICE void cp_async8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
MOE_DEVICE void fetch_wide(const Tensor& t, int64_t chunk, uint32_t slot) {
  // the chunk's place is the same for the block, a thread's in it a 32-bit offset
  const int64_t c0 = chunk * kChunk;
  const char* w = reinterpret_cast<const char*>((t.p_bf16 ? t.master : static_cast<float*>(t.p)) + c0);
  const uint32_t x = threadIdx.x, at = slot + x * 16u;
  if (t.g_bf16) {
    cp_async16(at, static_cast<const char*>(t.g) + c0 * 2 + x * 16u);
  } else {
    const char* g = static_cast<const char*>(t.g) + c0 * 4;
    cp_async16(at, g + x * 32u);
    cp_async16(at + 16 * kThreads, g + x * 32u + 16);
  }
  cp_async16(at + 32 * kThreads, w + x * 32u);
  cp_async16(at + 48 * kThreads, w + x * 32u + 16);
  const uint32_t codes = slot + 64 * kThreads + x * 8u;
  cp_async8(codes, static_cast<const char*>(t.m) + c0 + x * 8u);
  cp_async8(codes + 8 * kThreads, static_cast<const char*>(t.v) + c0 + x * 8u);
}

// A whole chunk of a tensor whose arrays allow whole vectors: a thread has eight elements. 8-bit
// states: from a slot that fetch_wide has filled, sm and sr the warp's
// scales, key that of the chunk's random words.
template <int BITS>
MOE_DEVICE void adamw_wide(const Tensor& t, int64_t chunk, const char* slot, uint32_t sm,
                           uint32_t sr, uint32_t key, const Now& n, const Step& s) {
  const int64_t c0 = chunk * kChunk;  // the same for the block
  const uint32_t x = threadIdx.x;
  char* weights = reinterpret_cast<char*>((t.p_bf16 ? t.master : static_cast<float*>(t.p)) + c0);
  char* state_m = static_cast<char*>(t.m) + c0 * (BITS / 8);
  char* state_v = static_cast<char*>(t.v) + c0 * (BITS / 8);
  float g[8], p[8], m[8], v[8];
  uint32_t gw[4];
  if constexpr (BITS == 8) {
    uint32_t mw[4], rw[4];
    const uint2* codes = reinterpret_cast<const uint2*>(slot + 64 * kThreads) + threadIdx.x;
    decode8<true>(codes[0], sm, mw);
    decode8<false>(codes[kThreads], sr, rw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[2 * i] = bf16_lo(mw[i]);
      m[2 * i + 1] = bf16_hi(mw[i]);
      v[2 * i] = bf16_lo(rw[i]);
      v[2 * i + 1] = bf16_hi(rw[i]);
    }
    const float4* q = reinterpret_cast<const float4*>(slot) + threadIdx.x;
    const float4 w0 = q[2 * kThreads], w1 = q[3 * kThreads], g0 = q[0];
    p[0] = w0.x; p[1] = w0.y; p[2] = w0.z; p[3] = w0.w;
    p[4] = w1.x; p[5] = w1.y; p[6] = w1.z; p[7] = w1.w;
    g[0] = g0.x; g[1] = g0.y; g[2] = g0.z; g[3] = g0.w;
    if (t.g_bf16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) gw[i] = __float_as_uint(g[i]);
    } else {
      const float4 g1 = q[kThreads];
      g[4] = g1.x; g[5] = g1.y; g[6] = g1.z; g[7] = g1.w;
    }
  } else {
    load8(state_m + x * 32u, m);
    load8(state_v + x * 32u, v);
    if (t.g_bf16) {
      const uint4 q = load4(static_cast<const char*>(t.g) + c0 * 2 + x * 16u);
      gw[0] = q.x;
      gw[1] = q.y;
      gw[2] = q.z;
      gw[3] = q.w;
    } else {
      load8(static_cast<const char*>(t.g) + c0 * 4 + x * 32u, g);
    }
    load8(weights + x * 32u, p);
  }
  if (t.g_bf16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[2 * i] = bf16_lo(gw[i]);
      g[2 * i + 1] = bf16_hi(gw[i]);
    }
  }
  const float lr_decay = n.lr * t.decay;
  float most_m = 0.f, most_r = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gs = __fmul_rn(g[j], n.factor);
    m[j] = __fadd_rn(__fmul_rn(m[j], s.b1), __fmul_rn(gs, s.c1));
    if constexpr (BITS == 8) v[j] = __fmul_rn(v[j], v[j]);
    v[j] = __fadd_rn(__fmul_rn(v[j], s.b2), __fmul_rn(__fmul_rn(gs, s.c2), gs));
    const float r = sqrt_approx(v[j]);
    // r rb + eps is between 2^-39 and 2^126 (moe_adamw_step's `vectors` and `far`)
    p[j] = (p[j] - p[j] * lr_decay) - n.a * (m[j] * rcp_approx(r * n.rb + s.eps));
    if constexpr (BITS == 8) {
      most_m = most_of(most_m, m[j]);
      most_r = most_of(most_r, r);
    }
  }
  store8(weights + x * 32u, p);
  if (t.p_bf16)
    *reinterpret_cast<uint4*>(static_cast<char*>(t.p) + c0 * 2 + x * 16u) =
        make_uint4(pack_bf16x2(p[0], p[1]), pack_bf16x2(p[2], p[3]), pack_bf16x2(p[4], p[5]),
                   pack_bf16x2(p[6], p[7]));
  if constexpr (BITS == 32) {
    store8(state_m + x * 32u, m);
    store8(state_v + x * 32u, v);
  } else {
    const uint2 scales =
        hold8(m, v, most_m, most_r, (uint32_t)c0 + x * 8u, key,
              reinterpret_cast<uint2*>(state_m + x * 8u), reinterpret_cast<uint2*>(state_v + x * 8u));
    if ((x & 31) == 0) {
      t.m_scale[chunk * kWarps + (x >> 5)] = (uint8_t)scales.x;
      t.v_scale[chunk * kWarps + (x >> 5)] = (uint8_t)scales.y;
    }
  }
}

// Any chunk: a warp's lane i has every 32nd element of its block of 256 from i on.
template <int BITS, bool FAR>
MOE_DEVICE void adamw_any(const Tensor& t, int64_t chunk, const Now& n, const Step& s) {
  const int lane = threadIdx.x & 31;
  const int64_t blk = chunk * kWarps + (threadIdx.x >> 5), e0 = blk * kBlock + lane;
  if (e0 - lane >= t.numel) return;
  float* weights = t.p_bf16 ? t.master : static_cast<float*>(t.p);
  const float lr_decay = n.lr * t.decay;
  uint32_t sm = 0, sv = 0, most_m = 0, most_r = 0;
  if constexpr (BITS == 8) {
    sm = t.m_scale[blk];
    sv = t.v_scale[blk];
  }
  float g[8], p[8], m[8], r[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t e = e0 + j * 32;
    g[j] = p[j] = m[j] = r[j] = 0.f;
    if (e >= t.numel) continue;
    g[j] = t.g_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.g)[e])
                    : static_cast<const float*>(t.g)[e];
    p[j] = weights[e];
    if constexpr (BITS == 8) {
      m[j] = decode_m(static_cast<const uint8_t*>(t.m)[e], sm);
      r[j] = decode_r(static_cast<const uint8_t*>(t.v)[e], sv);
    } else {
      m[j] = static_cast<const float*>(t.m)[e];
      r[j] = static_cast<const float*>(t.v)[e];
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t e = e0 + j * 32;
    const float v0 = BITS == 8 ? __fmul_rn(r[j], r[j]) : r[j];
    const Moments o = advance(__fmul_rn(g[j], n.factor), m[j], v0, s);
    m[j] = o.m;
    r[j] = o.r;
    if constexpr (BITS == 8) {  // elements past the end are 0
      most_m = max(most_m, __float_as_uint(fabsf(o.m)));
      most_r = max(most_r, __float_as_uint(fabsf(o.r)));
    }
    if (e >= t.numel) continue;
    const float w = update<FAR>(p[j], o, lr_decay, n, s);
    weights[e] = w;
    if (t.p_bf16) static_cast<__nv_bfloat16*>(t.p)[e] = __float2bfloat16_rn(w);
    if constexpr (BITS == 32) {
      static_cast<float*>(t.m)[e] = o.m;
      static_cast<float*>(t.v)[e] = o.v;
    }
  }
  if constexpr (BITS == 8) {
    sm = block_scale(__reduce_max_sync(0xFFFFFFFFu, most_m));
    sv = block_scale(__reduce_max_sync(0xFFFFFFFFu, most_r));
    const uint32_t key = word_key(t, e0, n);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t e = e0 + j * 32;
      if (e >= t.numel) continue;
      const uint32_t w = mix((uint32_t)e ^ key);
      const uint32_t c = encode(fabsf(m[j]), w & 0xFFFFu, sm, 127);
      static_cast<uint8_t*>(t.m)[e] = (uint8_t)(c | (c && m[j] < 0.f ? 128u : 0u));
      static_cast<uint8_t*>(t.v)[e] = (uint8_t)encode(r[j], w >> 16, sv, 255);
    }
    if (lane == 0) {
      t.m_scale[blk] = (uint8_t)sm;
      t.v_scale[blk] = (uint8_t)sv;
    }
  }
}

// 32-bit states: four blocks an SM (403 M elements, blocks that fit alone: 1740 us; three 1826,
// five 1903). 8-bit ones: three, as a fourth spills (101 M: 470 us against 502). FAR: an eps that
// only single elements and rounded quotients are right for, which the others do not pay for (fp32
// weights off the vectors' boundaries, 101 M: 440 us, 506 with them).
template <int BITS, bool FAR>
__global__ void __launch_bounds__(kThreads, BITS == 8 ? 3 : 4)
    adamw_kernel(const __grid_constant__ Batch b, const __grid_constant__ Step s) {
  MOE_GRIDDEP_ENTRY();
  int64_t c = blockIdx.x;
  int i = c < b.chunks ? find_tensor(b, c) : 0;
  auto wide = [](const Tensor& t, int64_t chunk) {
    return t.wide && (chunk + 1) * kChunk <= t.numel;
  };
  auto step_numbers = [&]() {
    __shared__ Now sn;
    step_now(s, sn);
    __syncthreads();
    return sn;
  };
  Now n;
  if constexpr (BITS == 32 || FAR) {
    n = step_numbers();
    if (n.skip) return;
    for (; c < b.chunks; c += gridDim.x) {
      while (i + 1 < b.n && b.t[i + 1].first <= c) ++i;
      const Tensor& t = b.t[i];
      const int64_t chunk = c - t.first;
      if constexpr (FAR) {
        adamw_any<BITS, true>(t, chunk, n, s);
      } else {
        if (wide(t, chunk)) adamw_wide<32>(t, chunk, nullptr, 0, 0, 0, n, s);
        else adamw_any<32, false>(t, chunk, n, s);
      }
    }
  } else {
    extern __shared__ __align__(16) char ring[];
    uint32_t sm = 0, sr = 0;
    auto fetch = [&](int turn) {  // of chunk c
      if (c < b.chunks) {
        while (i + 1 < b.n && b.t[i + 1].first <= c) ++i;
        const Tensor& t = b.t[i];
        const int64_t chunk = c - t.first;
        if (wide(t, chunk)) {
          fetch_wide(t, chunk, smem_u32(ring) + turn * kSlotBytes);
          sm = t.m_scale[chunk * kWarps + (threadIdx.x >> 5)];
          sr = t.v_scale[chunk * kWarps + (threadIdx.x >> 5)];
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    fetch(0);
    n = step_numbers();
    if (n.skip) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      return;
    }
    for (int turn = 0; c < b.chunks; turn ^= 1) {
      const Tensor& t = b.t[i];
      const int64_t chunk = c - t.first;
      const uint32_t m_scale = sm, r_scale = sr;
      c += gridDim.x;
      fetch(turn ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      if (wide(t, chunk))
        adamw_wide<8>(t, chunk, ring + turn * kSlotBytes, m_scale, r_scale,
                      word_key(t, chunk * kChunk, n), n, s);
      else
        adamw_any<8, false>(t, chunk, n, s);
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

// Elements a block reads back at a time: sixteen a thread, so that it writes whole 32-byte sectors
// (33.6 M elements 33 us; by sixteen bytes 43).
constexpr int kReadChunk = 2 * kChunk;
struct MomentsOut {
  __nv_bfloat16 *m[kCap], *v[kCap];
};
__global__ void __launch_bounds__(kThreads)
    adamw_moments_kernel(const __grid_constant__ Batch b, const __grid_constant__ MomentsOut out) {
  MOE_GRIDDEP_ENTRY();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const int i = find_tensor(b, c);
    const Tensor& t = b.t[i];
    const int64_t c0 = (c - t.first) * kReadChunk;
    if (t.wide && c0 + kReadChunk <= t.numel) {
      const int64_t e = c0 + threadIdx.x * 16;
      const uint32_t sm = t.m_scale[e / kBlock], sv = t.v_scale[e / kBlock];
      const uint4 cm = load4(static_cast<const uint8_t*>(t.m) + e);
      const uint4 cv = load4(static_cast<const uint8_t*>(t.v) + e);
      auto put = [&](__nv_bfloat16* to, auto sign, const uint4& q, uint32_t scale) {
        uint32_t lo[4], hi[4];
        decode8<sign.value>(make_uint2(q.x, q.y), scale, lo);
        decode8<sign.value>(make_uint2(q.z, q.w), scale, hi);
        const uint32_t w[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        st_global_v8(to + e, w);
      };
      put(out.m[i], std::true_type(), cm, sm);
      put(out.v[i], std::false_type(), cv, sv);
      continue;
    }
    for (int h = 0; h < kReadChunk / kChunk; ++h) {
      const int64_t e0 = c0 + h * kChunk + warp * kBlock;
      if (e0 >= t.numel) break;
      const uint32_t sm = t.m_scale[e0 / kBlock], sv = t.v_scale[e0 / kBlock];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t e = e0 + j * 32 + lane;
        if (e >= t.numel) continue;
        out.m[i][e] = __float2bfloat16_rn(decode_m(static_cast<const uint8_t*>(t.m)[e], sm));
        out.v[i][e] = __float2bfloat16_rn(decode_r(static_cast<const uint8_t*>(t.v)[e], sv));
      }
    }
  }
}

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Tensors [i, ..) of the list that hold elements, up to kCap; returns the next index. vectors:
// whole ones where the arrays allow.
int fill_batch(Batch& b, int i, int n, const moe_adamw_tensor_t* list, int bits, bool vectors,
               int chunk = kChunk) {
  b.n = 0;
  b.chunks = 0;
  const int state = bits == 8 ? 8 : 32;  // bytes of eight values
  for (; i < n && b.n < kCap; ++i) {
    const moe_adamw_tensor_t& l = list[i];
    if (l.numel == 0) continue;
    const int pb = l.param_dtype == MOE_DT_BF16, gb = l.grad_dtype == MOE_DT_BF16;
    const bool wide = vectors && on(l.param, pb ? 16 : 32) && on(l.master, 32) && on(l.grad, gb ? 16 : 32) &&
                      on(l.m, state) && on(l.v, state);
    b.t[b.n++] = {l.param, l.master, l.grad, l.m, l.v, l.m_scale, l.v_scale, l.numel, b.chunks,
                  l.decay, i, (int16_t)pb, (int16_t)gb, (int16_t)wide, 0};
    b.chunks += (l.numel + chunk - 1) / chunk;
  }
  return i;
}

// At most kTurns times the blocks that fit at once. Short blocks start at other times and so
// spread their reads, work and writes: 403 M elements with 32-bit states 1600 us at a chunk a
// block, 1752 with the blocks that fit alone; 101 M with 8-bit states, whose blocks fetch ahead
// and pay for their first chunk, 423 us with their moments at 16 turns, 455 at 4, 442 at 32, 592
// at a chunk a block (before the moments' last step, which took 28 us from each).
template <auto Kernel, int kSmem, int kTurns>
int adamw_blocks(int64_t chunks) {
  static DeviceCache cache;
  const int per_sm = std::max(1, cache.get(current_device(), [] {
    return blocks_per_sm(reinterpret_cast<const void*>(Kernel), kThreads, kSmem);
  }));
  const int64_t fit = (int64_t)std::max(device_sms(), 1) * per_sm * kTurns;
  return (int)std::max<int64_t>(1, std::min(chunks, fit));
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
  // an eps above 0 stays above it: a weight without gradients so far does not move (0 / eps)
  const float eps32 = eps > 0 ? std::max((float)eps, 0x1p-149f) : 0.f;
  Step step = {(float)lr, (float)beta1, (float)(1 - beta1), (float)beta2, (float)(1 - beta2),
               eps32, max_norm, std::log(beta1), std::log(beta2), lr_device, grad_norm,
               mix((uint32_t)seed ^ mix((uint32_t)(seed >> 32))),
               reinterpret_cast<unsigned long long*>(counters), 0};
  // The vectors' approximate root of a v below 2^-126 is 0 in the place of up to 2^-63. An eps
  // that loses that in its rounding hides it; under a smaller one every element takes the rounded
  // root, element by element: 101 M mixed weights at eps 1e-12 612 us against 403 at 1e-8 (8-bit
  // states 1040 against 297). r / sqrt(1 - beta2^t) is 0 or between 2^-75 and 2^91: a denominator outside the approximate
  // quotients' range comes from eps alone.
  const bool vectors = eps * 0x1p-24 >= 0x1p-63 / std::sqrt(1 - beta2);
  const bool far = (eps > 0 && eps < 0x1p-126) || eps > 0x1p125;
  Batch b;
  int i = 0;
  do {
    i = fill_batch(b, i, n, tensors, state_bits, vectors);
    int left = i;
    while (left < n && tensors[left].numel == 0) ++left;
    step.last = left == n;
    auto launch = [&](auto bits, auto is_far) {
      constexpr auto kernel = adamw_kernel<bits.value, is_far.value>;
      // 8-bit states fetch their next chunk ahead
      constexpr int smem = bits.value == 8 && !is_far.value ? kRingBytes : 0;
      constexpr int turns = smem ? 16 : 4096;
      return launch_pdl(kernel, adamw_blocks<kernel, smem, turns>(b.chunks), kThreads, smem, s, 1, b,
                        step);
    };
    using B8 = std::integral_constant<int, 8>;
    using B32 = std::integral_constant<int, 32>;
    const cudaError_t e = state_bits == 8 ? (far ? launch(B8(), std::true_type())
                                                 : launch(B8(), std::false_type()))
                                          : (far ? launch(B32(), std::true_type())
                                                 : launch(B32(), std::false_type()));
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
    i = fill_batch(b, i, n, tensors, 8, true, kReadChunk);
    if (b.n == 0) break;
    for (int j = 0; j < b.n; ++j) {
      out.m[j] = static_cast<__nv_bfloat16*>(m_out[b.t[j].index]);
      out.v[j] = static_cast<__nv_bfloat16*>(v_out[b.t[j].index]);
      b.t[j].wide = on(b.t[j].m, 16) && on(b.t[j].v, 16) && on(out.m[j], 32) && on(out.v[j], 32);
    }
    const int grid = adamw_blocks<adamw_moments_kernel, 0, 4096>(b.chunks);
    const cudaError_t e = launch_pdl(adamw_moments_kernel, grid, kThreads, 0, s, 1, b, out);
    count_launch(s, MOE_K_ADAMW_MOMENTS);
    if (e != cudaSuccess) return cuda_fail(e, "AdamW moments launch");
  }
  return MOE_OK;
}

}  // extern "C"
