// Packed fp32 pairs: two values in one 64-bit register.
#pragma once

#include "common.cuh"

namespace moe {

// add / sub / mul / fma of pairs are two independent IEEE fp32 operations (round to nearest even),
// so they give exactly the scalar results; but a product that is an addend is joined with the sum into
// an fma when it is compiled (measured), which product_f32x2 prevents.
MOE_DEVICE uint64_t pack_f32x2(float lo, float hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
  return d;
}
MOE_DEVICE float f32x2_lo(uint64_t v) { return __uint_as_float((uint32_t)v); }
MOE_DEVICE float f32x2_hi(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
MOE_DEVICE uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
MOE_DEVICE uint64_t sub_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
MOE_DEVICE uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
MOE_DEVICE uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// a b rounded by itself: an fma with an addend of -0 that the compiler does not know (a kernel's
// argument, in both halves).
MOE_DEVICE uint64_t product_f32x2(uint64_t a, uint64_t b, uint64_t minus_zero) {
  return fma_f32x2(a, b, minus_zero);
}

}  // namespace moe
