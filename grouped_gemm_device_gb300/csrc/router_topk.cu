// Choice of experts and the gradient of its weights (moe_router_topk_fwd / moe_router_topk_bwd in
// include/moegmm.h).
//
//   s = sigmoid(l) or softmax(l);  v = s + bias;  the best groups, their best k experts;
//   w = scale s, or scale s / sum of the chosen s
//
// Rows of more than 16 experts: a warp has a token; lane i holds the VPL neighbouring experts i
// VPL .., so that the lowest lane that holds a maximum holds the lowest index, and a tree over
// lanes adds neighbours first. Up to 16 experts: a thread has a token.
//
// The choice is bound by instructions and their latency, not by bytes. Some 620 instructions a token
// of 256 experts in 8 groups were counted, two thirds of the issue slots. As written, a round for each
// of the k + 1 largest takes some 20, scores 30, sorted lists 35, groups 60, weights 60, 365 together;
// the rest (loads, the loop, addresses, the tests of near values, spills, tokens chosen anew) was not
// told apart. 65536 x 256, top 8, sigmoid and bias (the bytes: 11 us): 58 us with 4 of 8 groups (231
// with exact scores and a search over eight values a round, 63 when twice as many tokens as need be
// were chosen anew), 41 without groups; softmax scores and bias, 4 of 8 groups 59 us, softmax
// probabilities without groups 46. Groups that are not whole lanes go by definition: 65536 x 160, 3 of
// 8 groups, top 6, 182 us by softmax, 211 by sigmoid and bias; 65536 x 192, 4 of 8, top 8, 229 us. A
// thread a token: 65536 x 8, top 2, 5.2 us; 65536 x 16, top 4, 9.0 us. 16384 x 128 bf16, top 4: 7.5 us,
// two launches; one token 4.0 us, the host's. The gradient writes a row a token, and reads one where it
// adds: 65536 x 256 added 32 us, 4.4 TB/s; of all probabilities 29 us, added 34.
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

// The VPL logits of a lane; NaN and what lies past E read as -inf. vec: rows lie on boundaries of
// VPL logits and E is a multiple of VPL.
template <int VPL, typename LT>
MOE_DEVICE void load_logits(const LT* row, int E, int lane, bool vec, float (&v)[VPL]) {
  const int e0 = lane * VPL;
  if constexpr (VPL * sizeof(LT) >= 4) {
   if (vec) {
    constexpr int W = VPL * sizeof(LT) / 4;
    uint32_t w[W];
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0xFFFFFFFFu;  // NaN
    if (e0 < E) {
      const LT* p = row + e0;
      if constexpr (W == 8)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4 % W]),
                       "=r"(w[5 % W]), "=r"(w[6 % W]), "=r"(w[7 % W])
                     : "l"(p));
      else if constexpr (W == 4)
        asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(w[0]), "=r"(w[1]), "=r"(w[2 % W]), "=r"(w[3 % W])
                     : "l"(p));
      else if constexpr (W == 2)
        asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1 % W]) : "l"(p));
      else
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      float x;
      if constexpr (sizeof(LT) == 4) x = __uint_as_float(w[j % W]);
      else x = (j & 1) ? bf16_hi(w[(j >> 1) % W]) : bf16_lo(w[(j >> 1) % W]);
      v[j] = fmaxf(x, -INFINITY);
    }
    return;
   }
  }
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = e0 + j;
    v[j] = e < E ? fmaxf(to_f(row[e]), -INFINITY) : -INFINITY;
  }
}

// VPL floats at a boundary of as many.
template <int VPL>
MOE_DEVICE void load_floats(const float* p, float (&v)[VPL]) {
  if constexpr (VPL == 8) {
    asm volatile("ld.global.L1::no_allocate.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]),
                   "=f"(v[6]), "=f"(v[7])
                 : "l"(p));
  } else if constexpr (VPL == 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x;
    v[1] = q.y;
    v[2] = q.z;
    v[3] = q.w;
  } else if constexpr (VPL == 2) {
    const float2 q = *reinterpret_cast<const float2*>(p);
    v[0] = q.x;
    v[1] = q.y;
  } else {
    v[0] = p[0];
  }
}
template <int VPL>
MOE_DEVICE void store_floats(float* p, const float (&v)[VPL]) {
  if constexpr (VPL == 8) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else if constexpr (VPL == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else if constexpr (VPL == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  } else {
    p[0] = v[0];
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

// The k experts of one token in lanes 0 .. k - 1, by definition: exact values, a round for each
// expert and group. `room`: two rows of 256 of the warp's shared memory. A call of its own: few
// tokens need it, and the others' registers and instructions stay few.
template <int VPL, typename LT>
__device__ __noinline__ int choose(const LT* row, const float* bias, const Choice& c,
                                   float (*room)[256]) {
  const int lane = threadIdx.x & 31;
  float x[VPL], v[VPL];
  load_logits<VPL>(row, c.E, lane, false, x);
  const bool by_score = bias || (c.n_group > 1 && c.group_top == 2);
#pragma unroll
  for (int j = 0; j < VPL; ++j) v[j] = x[j];
  if (by_score && c.score == MOE_SCORE_SIGMOID) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) v[j] = sigmoid(v[j]);
  } else if (by_score) {
    softmax_row<VPL>(v, c.E, lane);
  }
  uint32_t key[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane * VPL + j;
    if (bias && e < c.E) v[j] = __fadd_rn(v[j], fmaxf(bias[e], -INFINITY));
    key[j] = e < c.E ? ordered(bias ? v[j] : x[j]) : 0u;
  }
  if (c.n_group > 1) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      room[0][lane * VPL + j] = bias ? v[j] : x[j];
      room[1][lane * VPL + j] = v[j];
    }
    __syncwarp();
    const int size = c.E / c.n_group;
    float value[VPL];  // of groups lane, lane + 32, ..
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int grp = lane + 32 * j;
      float best = -INFINITY, next = -INFINITY;
      if (grp < c.n_group)
        for (int i = grp * size; i < (grp + 1) * size; ++i) {
          const float a = c.group_top == 1 ? room[0][i] : room[1][i];
          next = fmaxf(next, fminf(a, best));
          best = fmaxf(best, a);
        }
      value[j] = c.group_top == 1 ? best : fmaxf(__fadd_rn(best, next), -INFINITY);
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      room[0][lane + 32 * j] = value[j];
      room[1][lane + 32 * j] = 0.f;
    }
    __syncwarp();
    uint32_t gkey[VPL];  // a group a place, as the experts
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      gkey[j] = lane * VPL + j < c.n_group ? ordered(room[0][lane * VPL + j]) : 0u;
    for (int i = 0; i < c.topk_group; ++i) {
      const int grp = take_best<VPL>(gkey, lane);
      if (lane == 0) room[1][grp] = 1.f;
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (lane * VPL + j < c.E && room[1][(lane * VPL + j) / size] == 0.f) key[j] = 0;
    __syncwarp();
  }
  int mine = 0;
  for (int j = 0; j < c.k; ++j) {
    const int e = take_best<VPL>(key, lane);
    if (lane == j) mine = e;
  }
  return mine;
}

// Descending; the larger one of a pair first.
MOE_DEVICE void order_pair(float& a, float& b) {
  const float hi = fmaxf(a, b);
  b = fminf(a, b);
  a = hi;
}
MOE_DEVICE void sort4(float& a, float& b, float& c, float& d) {
  order_pair(a, b);
  order_pair(c, d);
  order_pair(a, c);
  order_pair(b, d);
  order_pair(b, c);
}
constexpr int list_of(int VPL) { return VPL < 5 ? VPL : 5; }
// A lane's largest values, descending: all of them, or the first five of eight (odd-even merge,
// Batcher 1968).
template <int VPL>
MOE_DEVICE void top_values(const float (&v)[VPL], float (&l)[list_of(VPL)]) {
  if constexpr (VPL <= 4) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) l[j] = v[j];
    if constexpr (VPL == 2) order_pair(l[0], l[1]);
    if constexpr (VPL == 4) sort4(l[0], l[1], l[2], l[3]);
  } else {
    float a[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = v[j];
    sort4(a[0], a[1], a[2], a[3]);
    sort4(a[4], a[5], a[6], a[7]);
#pragma unroll
    for (int j = 0; j < 4; ++j) order_pair(a[j], a[j + 4]);
    order_pair(a[2], a[4]);
    order_pair(a[3], a[5]);
    order_pair(a[1], a[2]);
    order_pair(a[3], a[4]);
    order_pair(a[5], a[6]);
#pragma unroll
    for (int j = 0; j < list_of(VPL); ++j) l[j] = a[j];
  }
}

// About 1 / (1 + exp(-x)): off by less than 2^-21.
MOE_DEVICE float sigmoid_near(float x) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}
// Whether a and b, a >= b, may be in another order than they seem, each being off by eps / 2 at
// most.
MOE_DEVICE bool near(float a, float b, float eps) { return !(a - b > eps) && b != -INFINITY; }

// A token's weights, one a lane below k (live): l the expert's logit, s its score (softmax alone).
MOE_DEVICE float weight_of(float l, float s, bool live, const Choice& c) {
  float w;
  if (c.score == MOE_SCORE_SIGMOID) {
    w = live ? sigmoid(l) : 0.f;
    if (c.renorm) w = __fdividef(w, sum8(w) + kWeightEps);
  } else if (c.renorm) {
    if (!live) l = -INFINITY;
    const float m = max8(l);
    w = live ? (l == m ? 1.0f : expf(l - m)) : 0.f;
    w = __fdividef(w, sum8(w));
  } else {
    w = s;
  }
  return w * c.scale;
}

// What decides the choice: the logits themselves; sigmoids (and biases), taken approximately;
// softmax probabilities.
enum Kind { kLogits = 0, kSigmoid = 1, kSoftmax = 2 };
constexpr float kFar = 3e38f;  // an infinite bias, and what lies past E, among approximate values

// GROUPS: the experts' groups are whole lanes, a power of two of them each. k <= KMAX. The choice
// goes by sorted lists, one a lane, whose heads the warp's maximum takes one by one. kSigmoid: 4
// instructions a score against some 17, and three bits of a value hold its place in the lane. A
// token with two deciding values too near to tell, with an infinite value among its k, or with a
// lane that holds equal ones or more than its list, is chosen anew by definition. Four blocks an SM,
// whose 64 registers spill 8 to 180 bytes with eight experts a lane, the most with groups and softmax:
// three, which spill at most 32, took 60.5 us in the place of 58.0 (65536 x 256, groups, sigmoid and
// bias), 61.1 of 59.2 (softmax and bias), 43.4 of 40.4 without groups.
template <int VPL, bool GROUPS, int KIND, int KMAX, typename LT>
__global__ void __launch_bounds__(kThreads, 4) router_topk_kernel(
    const LT* __restrict__ logits, int64_t ld, const float* __restrict__ bias,
    const uint8_t* __restrict__ mask, int T, const __grid_constant__ Choice c, int vec,
    int32_t* __restrict__ ids, float* __restrict__ weights, int32_t* __restrict__ counts) {
  MOE_GRIDDEP_ENTRY();
  constexpr int LIST = list_of(VPL);
  __shared__ int hist[256];
  __shared__ float room[kWarps][2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = c.E, k = c.k;
  if (counts) {
    for (int i = threadIdx.x; i < E; i += kThreads) hist[i] = 0;
    __syncthreads();
  }
  const int group_lanes = GROUPS ? E / c.n_group / VPL : 32;
  const int group = lane / group_lanes;
  // biases (0), and -inf past E
  float b[VPL], most = 0.f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    const int e = lane * VPL + j;
    b[j] = e >= E ? -INFINITY : KIND != kLogits && bias ? fmaxf(bias[e], -INFINITY) : 0.f;
    if (fabsf(b[j]) < INFINITY) most = fmaxf(most, fabsf(b[j]));
    if (KIND == kSigmoid) b[j] = fmaxf(fminf(b[j], kFar), -kFar);  // finite, for the place's bits
  }
  // kSigmoid: a value is off by 2^-21 in its score, by a step in the sum with its bias and by up
  // to seven in its last three bits, 2^-20 of it together; a sum of two (of up to 1 + the largest
  // bias) by twice that and a step of its own
  const float eps_group = 0x1p-19f + 0x1.2p-18f * (1.0f + warp_max(most));
  const uint32_t lane_bit = 1u << lane;
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  float x[VPL], next[VPL];
  if (t < T) load_logits<VPL>(logits + t * ld, E, lane, vec, next);
  for (; t < T; t += step) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) x[j] = next[j];
    if (t + step < T) load_logits<VPL>(logits + (t + step) * ld, E, lane, vec, next);
    if (mask && !mask[t]) {
      if (lane < k) {
        ids[t * k + lane] = -1;
        weights[t * k + lane] = 0.f;
      }
      continue;
    }
    const LT* row = logits + t * ld;
    float v[VPL], s[KIND == kSoftmax ? VPL : 1];  // values; probabilities
    if constexpr (KIND == kLogits) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) v[j] = x[j];
    } else if constexpr (KIND == kSigmoid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float y = sigmoid_near(x[j]) + b[j];
        v[j] = __uint_as_float((__float_as_uint(y) & ~(uint32_t)(VPL - 1)) | j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j) s[j] = x[j];
      softmax_row<VPL>(s, E, lane);
#pragma unroll
      for (int j = 0; j < VPL; ++j) v[j] = __fadd_rn(s[j], b[j]);
    }
    bool again = false, keep = true;
    if constexpr (GROUPS) {
      float best = -INFINITY, second = -INFINITY;
      if (c.group_top == 1) {
        if (KIND == kSoftmax && !bias) {
#pragma unroll
          for (int j = 0; j < VPL; ++j) best = fmaxf(best, x[j]);
        } else {
#pragma unroll
          for (int j = 0; j < VPL; ++j) best = fmaxf(best, v[j]);
        }
        for (int o = 1; o < group_lanes; o <<= 1)
          best = fmaxf(best, __shfl_xor_sync(kAll, best, o));
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          second = fmaxf(second, fminf(v[j], best));
          best = fmaxf(best, v[j]);
        }
        for (int o = 1; o < group_lanes; o <<= 1) {
          const float ob = __shfl_xor_sync(kAll, best, o), os = __shfl_xor_sync(kAll, second, o);
          second = fmaxf(fmaxf(second, os), fminf(best, ob));
          best = fmaxf(best, ob);
        }
        best = fmaxf(__fadd_rn(best, second), -INFINITY);
      }
      int before = 0;
#pragma unroll 4
      for (int i = 0; i < c.n_group; ++i) {
        const float other = __shfl_sync(kAll, best, i * group_lanes);
        before += other > best || (other == best && i < group);
      }
      keep = before < c.topk_group && group < c.n_group;
      if (KIND == kSigmoid) {
        const float in = -warp_max(keep ? -best : -INFINITY);
        const float out = warp_max(keep || group >= c.n_group ? -INFINITY : best);
        // sums with an infinite value are infinite, whatever else is in them
        again = near(in, out, eps_group) || !(fabsf(in) < 0.9f * kFar);
      }
    }
    if (KIND == kSoftmax && !bias) {  // the logits' order
#pragma unroll
      for (int j = 0; j < VPL; ++j) v[j] = x[j];
    }
    float list[LIST];
    top_values<VPL>(v, list);
    if (GROUPS && !keep) {
#pragma unroll
      for (int j = 0; j < LIST; ++j) list[j] = -INFINITY;
    }
    // round j's holder leaves the value and its lane
    float2* found = reinterpret_cast<float2*>(room[warp][0]);
    int pops = 0;
#pragma unroll
    for (int j = 0; j < KMAX + (KIND == kSigmoid); ++j) {
      const float m = warp_max(list[0]);
      const uint32_t who = __ballot_sync(kAll, list[0] == m);
      if ((who & (0u - who)) == lane_bit) {
        found[j] = make_float2(m, __int_as_float(lane));
#pragma unroll
        for (int i = 0; i + 1 < LIST; ++i) list[i] = list[i + 1];
        list[LIST - 1] = -INFINITY;
        if (VPL > LIST) ++pops;
      }
    }
    __syncwarp();
    const float2 mine_found = found[lane <= KMAX ? lane : 0];  // lane j: round j's
    const float taken = mine_found.x;
    const int from = __float_as_int(mine_found.y) & 31;
    __syncwarp();
    const float after = __shfl_down_sync(kAll, taken, 1);
    const int after_from = __shfl_down_sync(kAll, from, 1);
    again |= VPL > LIST && pops >= LIST;
    again |= lane < k && (KIND == kSigmoid ? !(fabsf(taken) < 0.9f * kFar) : taken == -INFINITY);
    int mine = 0;
    if constexpr (KIND == kSigmoid) {
      again |= lane < k &&
               near(taken, after, 0x1p-20f + 0x1p-19f * fmaxf(fabsf(taken), fabsf(after)));
      mine = from * VPL + (int)(__float_as_uint(taken) & (uint32_t)(VPL - 1));
    } else {
      again |= lane + 1 < k && taken == after && from == after_from;
#pragma unroll
      for (int j = VPL - 1; j >= 0; --j) {
        const float other = __shfl_sync(kAll, v[j], from);
        if (other == taken) mine = from * VPL + j;
      }
    }
    if (__any_sync(kAll, again)) mine = choose<VPL>(row, bias, c, room[warp]);
    const bool live = lane < k;
    const float l = live ? fmaxf(to_f(row[mine]), -INFINITY) : 0.f;
    float p = 0.f;
    if constexpr (KIND == kSoftmax) {
      if (!c.renorm) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
          const float other = __shfl_sync(kAll, s[j], mine / VPL);
          if (mine % VPL == j) p = other;
        }
      }
    }
    const float w = weight_of(l, p, live, c);
    if (live) {
      ids[t * k + lane] = mine;
      weights[t * k + lane] = w;
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

// Groups that are not whole lanes: every token by definition.
template <int VPL, typename LT>
__global__ void __launch_bounds__(kThreads) router_topk_any_kernel(
    const LT* __restrict__ logits, int64_t ld, const float* __restrict__ bias,
    const uint8_t* __restrict__ mask, int T, const __grid_constant__ Choice c,
    int vec, int32_t* __restrict__ ids, float* __restrict__ weights,
    int32_t* __restrict__ counts) {
  MOE_GRIDDEP_ENTRY();
  __shared__ int hist[256];
  __shared__ float room[kWarps][2][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = c.E, k = c.k;
  if (counts) {
    for (int i = threadIdx.x; i < E; i += kThreads) hist[i] = 0;
    __syncthreads();
  }
  for (int64_t t = (int64_t)blockIdx.x * kWarps + warp; t < T; t += (int64_t)gridDim.x * kWarps) {
    if (mask && !mask[t]) {
      if (lane < k) {
        ids[t * k + lane] = -1;
        weights[t * k + lane] = 0.f;
      }
      continue;
    }
    const LT* row = logits + t * ld;
    const int mine = choose<VPL>(row, bias, c, room[warp]);
    const bool live = lane < k;
    const float l = live ? fmaxf(to_f(row[mine]), -INFINITY) : 0.f;
    float p = 0.f;
    if (c.score == MOE_SCORE_SOFTMAX && !c.renorm) {
      float s[VPL];
      load_logits<VPL>(row, E, lane, false, s);
      softmax_row<VPL>(s, E, lane);
#pragma unroll
      for (int j = 0; j < VPL; ++j) {
        const float other = __shfl_sync(kAll, s[j], mine / VPL);
        if (mine % VPL == j) p = other;
      }
    }
    const float w = weight_of(l, p, live, c);
    if (live) {
      ids[t * k + lane] = mine;
      weights[t * k + lane] = w;
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

// Up to N experts without groups: a thread has a token.
template <int N, typename LT>
__global__ void __launch_bounds__(kThreads) router_topk_small_kernel(
    const LT* __restrict__ logits, int64_t ld, const float* __restrict__ bias,
    const uint8_t* __restrict__ mask, int T, const __grid_constant__ Choice c,
    int vec, int32_t* __restrict__ ids, float* __restrict__ weights,
    int32_t* __restrict__ counts) {
  MOE_GRIDDEP_ENTRY();
  __shared__ int hist[N];
  const int E = c.E, k = c.k;
  if (counts) {
    if (threadIdx.x < N) hist[threadIdx.x] = 0;
    __syncthreads();
  }
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < T;
       t += (int64_t)gridDim.x * kThreads) {
    if (mask && !mask[t]) {
      for (int j = 0; j < k; ++j) {
        ids[t * k + j] = -1;
        weights[t * k + j] = 0.f;
      }
      continue;
    }
    const LT* row = logits + t * ld;
    float x[N], s[N];
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      x[e] = e < E ? fmaxf(to_f(row[e]), -INFINITY) : -INFINITY;
      top = fmaxf(top, x[e]);
    }
    if (c.score == MOE_SCORE_SIGMOID) {
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] = sigmoid(x[e]);
    } else {
      float sum[N];
#pragma unroll
      for (int e = 0; e < N; ++e)
        sum[e] = s[e] = e >= E ? 0.f : x[e] == top ? 1.0f : expf(x[e] - top);
#pragma unroll
      for (int w = 1; w < N; w <<= 1)
#pragma unroll
        for (int e = 0; e < N; e += 2 * w) sum[e] = __fadd_rn(sum[e], sum[e + w]);
      const float inv = __frcp_rn(sum[0]);
#pragma unroll
      for (int e = 0; e < N; ++e) s[e] = __fmul_rn(s[e], inv);
    }
    uint32_t left = E < 32 ? (1u << E) - 1u : ~0u;
    float w[8], total = 0.f, first = 0.f;
    int id[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= k) break;
      float best = -INFINITY;
      int at = -1;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float v = bias ? __fadd_rn(s[e], e < E ? fmaxf(bias[e], -INFINITY) : 0.f) : x[e];
        if ((left >> e & 1u) && (at < 0 || v > best)) {
          best = v;
          at = e;
        }
      }
      left &= ~(1u << at);
      float l = 0.f, sc = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (e == at) {
          l = x[e];
          sc = s[e];
        }
      id[j] = at;
      w[j] = c.renorm && c.score == MOE_SCORE_SOFTMAX ? l : sc;
      first = j == 0 ? w[j] : fmaxf(first, w[j]);
    }
    if (c.renorm) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (j >= k) break;
        if (c.score == MOE_SCORE_SOFTMAX) w[j] = w[j] == first ? 1.0f : expf(w[j] - first);
        total += w[j];
      }
      if (c.score == MOE_SCORE_SIGMOID) total += kWeightEps;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= k) break;
      ids[t * k + j] = id[j];
      weights[t * k + j] = (c.renorm ? w[j] / total : w[j]) * c.scale;
      if (counts) atomicAdd(&hist[id[j]], 1);
    }
  }
  if (!counts) return;
  __syncthreads();
  if (threadIdx.x < E) {
    const int n = hist[threadIdx.x];
    if (gridDim.x == 1) counts[threadIdx.x] = n;
    else if (n) atomicAdd(&counts[threadIdx.x], n);
  }
}

// s (1 - s) from l, q = exp(-l) and s = 1 / (1 + q), without a difference of near numbers.
MOE_DEVICE float slope_of(float l, float q, float s) {
  return l >= 0.f ? q * s * s : s * (1.0f - s);
}
// What a token's slot, one a lane below 8 (-inf and 0 in the others), adds to its expert's
// gradient. l, u: the slot's logit and scale * d_weight, e its expert or -1.
MOE_DEVICE float slot_grad(float l, float u, int e, int score, int renorm) {
  if (score == MOE_SCORE_SIGMOID) {
    const float q = expf(-l), s = __frcp_rn(1.0f + q);
    if (renorm) {
      const float sc = e >= 0 ? s : 0.f, total = sum8(sc) + kWeightEps;
      u = (u - sum8(__fmul_rn(u, sc)) / total) / total;
    }
    u *= slope_of(l, q, s);
  } else if (renorm) {
    const float m = max8(l);
    float w = e >= 0 ? (l == m ? 1.0f : expf(l - m)) : 0.f;
    w = w / fmaxf(sum8(w), 1.0f);  // at least the maximum's 1, but for a token without slots
    u = w * (u - sum8(w * u));
  }
  return e < 0 ? 0.f : u;
}

// A warp has a token: its lanes 0 .. k - 1 the slots' parts, which reach the experts through a row
// of shared memory; each lane then has the VPL experts it owns. WHOLE: every probability has a
// gradient.
template <int VPL, bool VEC, bool WHOLE, typename LT>
__global__ void __launch_bounds__(kThreads) router_topk_grad_kernel(
    const LT* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, int T, int E, int k, int score, int renorm, float scale,
    const float* add_to, int64_t ld_add, float* d, int64_t ldd) {
  MOE_GRIDDEP_ENTRY();
  __shared__ __align__(32) float rows[kWarps][256];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* row_c = rows[warp];
  for (int i = lane; i < 256; i += 32) row_c[i] = 0.f;
  __syncwarp();
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t t = (int64_t)blockIdx.x * kWarps + warp;
  int e_next = -1;
  float u_next = 0.f;
  auto slot_of = [&](int64_t row) {
    e_next = -1;
    u_next = 0.f;
    if (row < T && lane < k) {
      e_next = ids[row * k + lane];
      u_next = dw[row * k + lane];
    }
  };
  slot_of(t);
  for (; t < T; t += step) {
    int e = e_next >= 0 && e_next < E ? e_next : -1;
    float u = e >= 0 ? u_next * scale : 0.f, l = -INFINITY;
    const LT* row = logits + t * ld;
    if (!WHOLE && e >= 0) l = fmaxf(to_f(row[e]), -INFINITY);
    slot_of(t + step);
    float o[VPL], base[VPL];
    const int e0 = lane * VPL;
#pragma unroll
    for (int j = 0; j < VPL; ++j) base[j] = 0.f;
    if (add_to) {
      const float* from = add_to + t * ld_add + e0;
      if (VEC) {
        if (e0 < E) load_floats<VPL>(from, base);
      } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
          if (e0 + j < E) base[j] = from[j];
      }
    }
    if (!WHOLE) u = slot_grad(l, u, e, score, renorm);
    // slots that share an expert, which a mark left there by each shows, are added in their order
    if (e >= 0) row_c[e] = __int_as_float(lane);
    __syncwarp();
    const bool shared = e >= 0 && __float_as_int(row_c[e]) != lane;
    if (!__any_sync(kAll, shared)) {
      if (e >= 0) row_c[e] = u;
    } else {
      __syncwarp();
      if (e >= 0) row_c[e] = 0.f;
      __syncwarp();
      for (int i = 0; i < k; ++i) {
        if (lane == i && e >= 0) row_c[e] += u;
        __syncwarp();
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < VPL; ++j) o[j] = row_c[e0 + j];
    __syncwarp();
    if (e >= 0) row_c[e] = 0.f;
    if (WHOLE) {
      float p[VPL], a = 0.f;
      load_logits<VPL>(row, E, lane, VEC, p);
      softmax_row<VPL>(p, E, lane);
#pragma unroll
      for (int j = 0; j < VPL; ++j) a += p[j] * o[j];
#pragma unroll
      for (int q = 16; q > 0; q >>= 1) a += __shfl_xor_sync(kAll, a, q);
#pragma unroll
      for (int j = 0; j < VPL; ++j) o[j] = p[j] * (o[j] - a);
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j) o[j] += base[j];
    float* to = d + t * ldd + e0;
    if (VEC) {
      if (e0 < E) store_floats<VPL>(to, o);
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (e0 + j < E) to[j] = o[j];
    }
    __syncwarp();
  }
}

// Up to N experts: a thread has a token.
template <int N, typename LT>
__global__ void __launch_bounds__(kThreads) router_topk_grad_small_kernel(
    const LT* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const float* __restrict__ dw, int T, int E, int k, int score, int renorm, float scale,
    const float* add_to, int64_t ld_add, float* d, int64_t ldd) {
  MOE_GRIDDEP_ENTRY();
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < T;
       t += (int64_t)gridDim.x * kThreads) {
    const LT* row = logits + t * ld;
    float x[N], top = -INFINITY;  // of all experts, or (softmax, renorm) of the chosen ones
#pragma unroll
    for (int e = 0; e < N; ++e) {
      x[e] = e < E ? fmaxf(to_f(row[e]), -INFINITY) : -INFINITY;
      top = fmaxf(top, x[e]);
    }
    int id[8];
    float u[8], l[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      id[j] = -1;
      u[j] = 0.f;
      l[j] = -INFINITY;
      if (j < k) {
        const int e = ids[t * k + j];
        if (e >= 0 && e < E) {
          id[j] = e;
          u[j] = dw[t * k + j] * scale;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (i == e) l[j] = x[i];
        }
      }
    }
    float o[N];
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] = 0.f;
    const bool whole = score == MOE_SCORE_SOFTMAX && !renorm;
    if (!whole) {
      float s[8], slope[8], total = 0.f, dot = 0.f;
      if (score == MOE_SCORE_SOFTMAX) {
        top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, l[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (score == MOE_SCORE_SIGMOID) {
          const float q = expf(-l[j]);
          s[j] = __frcp_rn(1.0f + q);
          slope[j] = slope_of(l[j], q, s[j]);
        } else {
          s[j] = l[j] == top ? 1.0f : expf(l[j] - top);
          slope[j] = 0.f;
        }
        if (id[j] < 0) s[j] = 0.f;
        total += s[j];
        dot += __fmul_rn(u[j], s[j]);
      }
      if (score == MOE_SCORE_SIGMOID) total += kWeightEps;
      else total = fmaxf(total, 1.0f);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (renorm) u[j] = (u[j] - dot / total) / total;
        u[j] *= score == MOE_SCORE_SIGMOID ? slope[j] : s[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e)
        if (id[j] == e) o[e] += u[j];
    if (whole) {
      float total = 0.f, dot = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        x[e] = e >= E ? 0.f : x[e] == top ? 1.0f : expf(x[e] - top);
        total += x[e];
        dot += x[e] * o[e];
      }
      const float inv = 1.0f / total;
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] = x[e] * inv * (o[e] - dot * inv);
    }
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (e < E) d[t * ldd + e] = add_to ? add_to[t * ld_add + e] + o[e] : o[e];
  }
}

__global__ void __launch_bounds__(256) zero_counts_kernel(int32_t* counts, int E) {
  MOE_GRIDDEP_ENTRY();
  if ((int)threadIdx.x < E) counts[threadIdx.x] = 0;
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
int experts_a_lane(int E) { return E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : 8; }
// Calls fn with the experts a thread (4, 8 or 16) and a value of the logits' type.
template <class F>
void with_small(int E, int32_t dtype, F&& fn) {
  auto typed = [&](auto n) {
    if (dtype == MOE_DT_FP32) fn(n, float());
    else fn(n, __nv_bfloat16());
  };
  if (E <= 4) typed(I<4>());
  else if (E <= 8) typed(I<8>());
  else typed(I<16>());
}
constexpr int kSmall = 16;  // experts of a token that a thread has

// `per_block` tokens at a time a block, `per_sm` blocks an SM at most.
int topk_blocks(int64_t T, int per_block, int per_sm) {
  return (int)std::max<int64_t>(1, std::min<int64_t>((T + per_block - 1) / per_block,
                                                     (int64_t)std::max(device_sms(), 1) * per_sm));
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
  const bool small = E <= kSmall && n_group == 1;
  // as many as fit at once (three of router_topk_any_kernel above 128 experts: 65536 x 160 182 us,
  // with a grid of three an SM 144)
  const int grid = topk_blocks(T, small ? kThreads : kWarps, 4);
  cudaError_t e = cudaSuccess;
  if (T == 0 || grid > 1) {  // a single block writes the counts, several add to them
    if (counts) {
      e = launch_pdl(zero_counts_kernel, 1, 256, 0, s, 1, counts, E);
      count_launch(s, MOE_K_ROUTER_TOPK);
      if (e != cudaSuccess) return cuda_fail(e, "router counts launch");
    }
    if (T == 0) return MOE_OK;
  }
  const Choice c = {E, k, score, n_group, topk_group, group_top, renorm != 0, scale};
  const int vpl = experts_a_lane(E), size = E / n_group, lanes = size / vpl;
  const bool whole = size % vpl == 0 && (lanes & (lanes - 1)) == 0;  // groups of whole lanes
  const bool vec = E % vpl == 0 && ld_logits % vpl == 0 &&
                   on(logits, vpl * (logits_dtype == MOE_DT_FP32 ? 4 : 2));
  const bool by_score = bias || (n_group > 1 && group_top == 2);
  auto launch = [&](auto kernel, auto lt) {
    e = launch_pdl(kernel, grid, kThreads, 0, s, 1, static_cast<const decltype(lt)*>(logits),
                   ld_logits, bias, token_mask, T, c, (int)vec, topk_ids, topk_weights, counts);
  };
  if (small) {
    with_small(E, logits_dtype, [&](auto n, auto lt) {
      launch(router_topk_small_kernel<n.value, decltype(lt)>, lt);
    });
  } else if (n_group > 1 && !whole) {
    with_shape(E, logits_dtype, [&](auto v, auto lt) {
      launch(router_topk_any_kernel<v.value, decltype(lt)>, lt);
    });
  } else {
    with_shape(E, logits_dtype, [&](auto v, auto lt) {
      using LT = decltype(lt);
      constexpr int V = v.value;
      auto kind = [&](auto g, auto kmax) {
        constexpr bool G = g.value;
        constexpr int K = kmax.value;
        if (score == MOE_SCORE_SOFTMAX && (by_score || !renorm))
          launch(router_topk_kernel<V, G, kSoftmax, K, LT>, lt);
        else if (by_score) launch(router_topk_kernel<V, G, kSigmoid, K, LT>, lt);
        else launch(router_topk_kernel<V, G, kLogits, K, LT>, lt);
      };
      if (n_group > 1) kind(std::true_type(), I<8>());
      else if (k <= 4) kind(std::false_type(), I<4>());
      else kind(std::false_type(), I<8>());
    });
  }
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
  const Span sd = span(d_logits, E, ld_d, 4);
  if (spoils(sd, span(add_to, E, ld_add, 4), T) ||
      spoils(sd, span(logits, E, ld_logits, logits_dtype == MOE_DT_FP32 ? 4 : 2), T))
    return fail(MOE_ERR_INVALID_ARG, "d_logits shares memory with other rows of add_to or logits");
  if (!on(logits, logits_dtype == MOE_DT_FP32 ? 4 : 2) || !on(topk_ids, 4) || !on(d_weights, 4) ||
      !on(add_to, 4) || !on(d_logits, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (T == 0) return MOE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const bool small = E <= kSmall, whole = score == MOE_SCORE_SOFTMAX && !renorm;
  auto launch = [&](auto kernel, auto lt) {
    e = launch_pdl(kernel, topk_blocks(T, small ? kThreads : kWarps, 8), kThreads, 0, s, 1,
                   static_cast<const decltype(lt)*>(logits), ld_logits, topk_ids, d_weights, T, E,
                   k, score, (int)(renorm != 0), scale, add_to, ld_add, d_logits, ld_d);
  };
  const int vpl = experts_a_lane(E);
  const bool vec = E % vpl == 0 && ld_logits % vpl == 0 && ld_d % vpl == 0 &&
                   on(logits, vpl * (logits_dtype == MOE_DT_FP32 ? 4 : 2)) &&
                   on(d_logits, vpl * 4) && (!add_to || (ld_add % vpl == 0 && on(add_to, vpl * 4)));
  if (small) {
    with_small(E, logits_dtype, [&](auto n, auto lt) {
      launch(router_topk_grad_small_kernel<n.value, decltype(lt)>, lt);
    });
  } else {
    with_shape(E, logits_dtype, [&](auto v, auto lt) {
      using LT = decltype(lt);
      constexpr int V = v.value;
      if (vec && whole) launch(router_topk_grad_kernel<V, true, true, LT>, lt);
      else if (vec) launch(router_topk_grad_kernel<V, true, false, LT>, lt);
      else if (whole) launch(router_topk_grad_kernel<V, false, true, LT>, lt);
      else launch(router_topk_grad_kernel<V, false, false, LT>, lt);
    });
  }
  count_launch(s, MOE_K_ROUTER_TOPK_GRAD);
  if (e != cudaSuccess) return cuda_fail(e, "router top-k gradient launch");
  return MOE_OK;
}

}  // extern "C"
