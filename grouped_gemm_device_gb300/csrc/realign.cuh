// Bytes off 16-byte boundaries: rows whose stride is not a multiple of 16 bytes are read and
// written in the aligned 16-byte blocks that they straddle, and the bytes moved in registers (three
// conditional moves by 8, 4 and 2 bytes). An aligned block that holds a wanted byte lies in the
// same allocation as that byte.
#pragma once

#include "common.cuh"

namespace moe {

// Drops the first `lead` bytes (even, 0..14) of the 4 W: w[0 .. W - 5] holds those that follow.
template <int W>
MOE_DEVICE void drop_bytes(uint32_t (&w)[W], int lead) {
  if (lead & 8) {
#pragma unroll
    for (int k = 0; k < W - 2; ++k) w[k] = w[k + 2];
  }
  if (lead & 4) {
#pragma unroll
    for (int k = 0; k < W - 3; ++k) w[k] = w[k + 1];
  }
  if (lead & 2) {
#pragma unroll
    for (int k = 0; k < W - 4; ++k) w[k] = __funnelshift_r(w[k], w[k + 1], 16);
  }
}
// The other way: w[4..7] becomes the 16 bytes that start `lead` bytes before it.
MOE_DEVICE void keep_bytes(uint32_t (&w)[8], int lead) {
  if (lead & 8) {
#pragma unroll
    for (int k = 7; k >= 2; --k) w[k] = w[k - 2];
  }
  if (lead & 4) {
#pragma unroll
    for (int k = 7; k >= 3; --k) w[k] = w[k - 1];
  }
  if (lead & 2) {
#pragma unroll
    for (int k = 7; k >= 4; --k) w[k] = __funnelshift_l(w[k - 1], w[k], 16);
  }
}
// Zeros past the first `bytes` (even) of 16.
MOE_DEVICE void zero_past(uint32_t* w, int bytes) {
  if (bytes >= 16) return;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int left = bytes - 4 * k;
    w[k] = left >= 4 ? w[k] : left == 2 ? w[k] & 0xFFFFu : 0u;
  }
}
MOE_DEVICE int lead_bytes(const void* p) {
  return (int)(reinterpret_cast<uintptr_t>(p) & 15u);
}
// The first `bytes` (even, 1 or more; at most 16 count) bytes at p, zeros after them.
MOE_DEVICE uint4 load16_any(const void* p, int64_t bytes) {
  const int lead = lead_bytes(p), n = (int)(bytes < 16 ? bytes : 16);
  const uint4* base = reinterpret_cast<const uint4*>(static_cast<const char*>(p) - lead);
  const uint4 a = base[0], b = lead + n > 16 ? base[1] : make_uint4(0, 0, 0, 0);
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  drop_bytes(w, lead);
  zero_past(w, n);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace moe
