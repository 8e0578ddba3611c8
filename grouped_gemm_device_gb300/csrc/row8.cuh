// Rows of bf16 or fp32 elements in vectors of eight, on or off the vectors' boundaries.
//
// A vector is 16 bytes of bf16 or 32 of fp32. Rows off the boundaries (ANY) are read and written
// in the aligned vectors that they straddle: with `lead` the place of a row's first element in its
// first vector, element j of vector b is column 8 b - lead + j. What a row's first and last vector
// hold of other rows is cleared when read and left alone when written. An aligned vector that
// holds a wanted element lies in the same allocation as that element.
#pragma once

#include "realign.cuh"

namespace moe {

template <typename T>
MOE_DEVICE float to_float(T v) {
  if constexpr (sizeof(T) == 2) return __bfloat162float(v);
  else return v;
}
template <typename T>
MOE_DEVICE T from_float(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  static constexpr int kWords = 2 * sizeof(T);
  uint32_t w[kWords];
};
template <typename T>
MOE_DEVICE void zero8(Raw8<T>& r) {
#pragma unroll
  for (uint32_t& w : r.w) w = 0u;
}
// Streamed data is not kept in L1, which the weights of the following rows want.
template <typename T>
MOE_DEVICE void load8(const T* p, Raw8<T>& r) {
  if constexpr (sizeof(T) == 2)
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p));
  else
    asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]),
                   "=r"(r.w[5]), "=r"(r.w[6]), "=r"(r.w[7])
                 : "l"(p));
}
template <typename T>
MOE_DEVICE float at8(const Raw8<T>& r, int j) {  // j is a constant after unrolling
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[j]);
  else return (j & 1) ? bf16_hi(r.w[j >> 1]) : bf16_lo(r.w[j >> 1]);
}
// Zeros before element lo and from element hi on.
template <typename T>
MOE_DEVICE void clear8(Raw8<T>& r, int lo, int hi) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= lo && j < hi) continue;
    if constexpr (sizeof(T) == 4) r.w[j] = 0u;
    else r.w[j >> 1] &= (j & 1) ? 0x0000FFFFu : 0xFFFF0000u;
  }
}
// Rounded to T.
template <typename T>
MOE_DEVICE void round8(const float (&v)[8], Raw8<T>& r) {
#pragma unroll
  for (int k = 0; k < Raw8<T>::kWords; ++k)
    r.w[k] = sizeof(T) == 2 ? pack_bf16x2(v[(2 * k) & 7], v[(2 * k + 1) & 7])
                            : __float_as_uint(v[k & 7]);
}
// Stores the elements [lo, hi) of the vector at p.
template <bool ANY, typename T>
MOE_DEVICE void store8(T* p, const Raw8<T>& r, int lo, int hi) {
  if (!ANY || (lo <= 0 && hi >= 8)) {
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint4*>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else
      st_global_v8(p, r.w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= lo && j < hi) {
        if constexpr (sizeof(T) == 2)
          reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(r.w[j >> 1] >> (16 * (j & 1)));
        else
          reinterpret_cast<uint32_t*>(p)[j] = r.w[j];
      }
  }
}
template <typename T>
MOE_DEVICE int lead8(const T* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) / sizeof(T) & 7u);
}

// A norm's weights: bf16, fp32 or none (1); vec: on a vector's boundary.
struct Weight {
  const void* p;
  int16_t fp32, vec;
};
MOE_DEVICE float weight_at(const Weight& w, int64_t c) {
  if (!w.p) return 1.0f;
  return w.fp32 ? static_cast<const float*>(w.p)[c]
                : __bfloat162float(static_cast<const __nv_bfloat16*>(w.p)[c]);
}
// Those of columns c .. c + 7, zeros outside [0, N). ANY: c is any column from -7 on; otherwise a
// multiple of eight within N, and vec is set.
template <bool ANY>
MOE_DEVICE void weights8(const Weight& w, int c, int N, float (&v)[8]) {
  if (!w.p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.0f;
    return;
  }
  if (ANY && !w.vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j >= 0 && c + j < N ? weight_at(w, c + j) : 0.f;
    return;
  }
  const uint4* q = static_cast<const uint4*>(w.p);
  if (w.fp32) {
    const int b = ANY ? (c + 8) / 4 - 2 : c / 4;  // the 16 bytes of c, rounded down
    uint32_t u[12];
#pragma unroll
    for (int i = 0; i < (ANY ? 3 : 2); ++i) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (!ANY || (b + i >= 0 && (b + i) * 4 < N)) x = __ldg(q + b + i);
      u[4 * i] = x.x;
      u[4 * i + 1] = x.y;
      u[4 * i + 2] = x.z;
      u[4 * i + 3] = x.w;
    }
    if (ANY) drop_bytes(u, (c - 4 * b) * 4);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(u[j]);
  } else {
    const int b = ANY ? (c + 8) / 8 - 1 : c / 8;
    uint32_t u[8];
#pragma unroll
    for (int i = 0; i < (ANY ? 2 : 1); ++i) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (!ANY || (b + i >= 0 && (b + i) * 8 < N)) x = __ldg(q + b + i);
      u[4 * i] = x.x;
      u[4 * i + 1] = x.y;
      u[4 * i + 2] = x.z;
      u[4 * i + 3] = x.w;
    }
    if (ANY) drop_bytes(u, (c - 8 * b) * 2);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = (j & 1) ? bf16_hi(u[j >> 1]) : bf16_lo(u[j >> 1]);
  }
  if (ANY && (c < 0 || c + 8 > N)) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < 0 || c + j >= N) v[j] = 0.f;
  }
}

// Sum over the G threads of a row's group: a warp, or a whole block, whose warps all add the warps'
// sums in the same order. `sm` must not be in use by a call less than one barrier ago.
template <int G>
MOE_DEVICE float group_sum(float a, float (&sm)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  if constexpr (G > 32) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) sm[threadIdx.x >> 5] = a;
    __syncthreads();
    if constexpr (G <= 256) {
      a = sm[0];
#pragma unroll
      for (int w = 1; w < G / 32; ++w) a += sm[w];
    } else {
      a = lane < G / 32 ? sm[lane] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    }
  }
  return a;
}

}  // namespace moe
