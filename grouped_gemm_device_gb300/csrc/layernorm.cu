// Layer norm over the last dimension, forward and backward (moe_layernorm_fwd /
// moe_layernorm_bwd in include/moegmm.h).
//
//   y = (x - mean) rstd gamma + beta;  h = (x - mean) rstd, u = dy gamma:
//   dx = rstd (u - mean_n(u) - h mean_n(u h));  dgamma = sum_m dy h;  dbeta = sum_m dy
//
// Bound by HBM: the forward reads and writes M N elements once, the backward reads x and dy and
// writes dx once. A row stays in registers between its statistics and its use, so the variance is
// taken about the mean (two passes over registers, not E[x^2] - mean^2). Statistics, sums and the
// weight-gradient partials are fp32. Widening bf16 runs at half the rate of the products, so it is
// done once a value where the registers allow.
#include "kernels.cuh"

namespace moe {
namespace {

// Backward blocks at most (rows of the partial weight gradients), by the row's length: short rows
// leave small partials and run more blocks.
constexpr int64_t kShortRow = 1024;
int64_t max_parts(int64_t N) { return N <= kShortRow ? 960 : 480; }

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

// VEC consecutive elements as they lie in memory: 16 bytes, or one element (VEC = 1).
template <typename T, int VEC>
struct Raw {
  uint32_t w[VEC == 1 ? 1 : 4];
  static_assert(VEC == 1 || VEC * sizeof(T) == 16, "one element or 16 bytes");
};
template <typename T, int VEC>
MOE_DEVICE void zero_raw(Raw<T, VEC>& r) {
#pragma unroll
  for (uint32_t& w : r.w) w = 0u;
}
// Streamed data is not kept in L1, which the weights of the following rows want.
template <typename T, int VEC>
MOE_DEVICE void load_raw(const T* p, Raw<T, VEC>& r) {
  if constexpr (VEC > 1) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
                 : "l"(p));
  } else if constexpr (sizeof(T) == 2) {
    r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else {
    r.w[0] = __float_as_uint(*p);
  }
}
template <typename T, int VEC>
MOE_DEVICE float raw_at(const Raw<T, VEC>& r, int j) {  // j is a constant after unrolling
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[j]);
  else return (j & 1) ? bf16_hi(r.w[j >> 1]) : bf16_lo(r.w[j >> 1]);
}

// VEC consecutive elements (VEC * sizeof(T) a multiple of 16 bytes, or VEC = 1) as fp32.
template <typename T, int VEC>
MOE_DEVICE void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = to_f(__ldg(p));
  } else {
    constexpr int W = VEC * sizeof(T) / 16;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint4 q = __ldg(reinterpret_cast<const uint4*>(p) + w);
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
  } else if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}

MOE_DEVICE float warp_sum(float a) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
  return a;
}
// Sum over the G threads of a row's group: a warp, or a whole block, whose warps all add the
// warps' sums in the same order. `sm` must not be in use by a call less than one barrier ago.
template <int G>
MOE_DEVICE float row_sum(float a, float (&sm)[32]) {
  a = warp_sum(a);
  if constexpr (G > 32) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) sm[threadIdx.x >> 5] = a;
    __syncthreads();
    if constexpr (G <= 256) {
      a = sm[0];
#pragma unroll
      for (int w = 1; w < G / 32; ++w) a += sm[w];
    } else {
      a = warp_sum(lane < G / 32 ? sm[lane] : 0.f);
    }
  }
  return a;
}
// Two sums at once; a block's calls take turns (0, 1, 0, ..) with the halves of `sm`.
template <int G>
MOE_DEVICE void row_sum2(float& a, float& b, float (&sm)[2][2][32], int turn) {
  a = warp_sum(a);
  b = warp_sum(b);
  if constexpr (G > 32) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (lane == 0) {
      sm[turn][0][w] = a;
      sm[turn][1][w] = b;
    }
    __syncthreads();
    if constexpr (G <= 256) {
      a = sm[turn][0][0];
      b = sm[turn][1][0];
#pragma unroll
      for (int i = 1; i < G / 32; ++i) {
        a += sm[turn][0][i];
        b += sm[turn][1][i];
      }
    } else {
      a = warp_sum(lane < G / 32 ? sm[turn][0][lane] : 0.f);
      b = warp_sum(lane < G / 32 ? sm[turn][1][lane] : 0.f);
    }
  }
}

// G threads (a warp of four in a block, or a whole block) take RP rows, PER vectors of VEC elements
// a thread and row: N <= G * PER * VEC. Two rows share each load of the weights.
template <typename XT, typename WT, int VEC, int G, int PER, int RP>
__global__ void __launch_bounds__(G < 128 ? 128 : G) ln_fwd_kernel(
    const XT* x, int64_t ldx, const WT* __restrict__ gamma, const WT* __restrict__ beta, XT* y,
    int64_t ldy, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t M, int N,
    float eps) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[2][RP][32];
  constexpr int R = (G < 128 ? 128 : G) / G;  // groups a block
  const int t = threadIdx.x % G;
  const int64_t row0 = ((int64_t)blockIdx.x * R + threadIdx.x / G) * RP;
  if (G == 32 && row0 >= M) return;  // a block's groups are its warps; otherwise R = 1
  Raw<XT, VEC> raw[RP][PER];
#pragma unroll
  for (int k = 0; k < RP; ++k)
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC;
      zero_raw(raw[k][i]);
      if (c < N && (RP == 1 || row0 + k < M)) load_raw(x + (row0 + k) * ldx + c, raw[k][i]);
    }
  float v[RP][PER][VEC], rstd[RP];
#pragma unroll
  for (int k = 0; k < RP; ++k) {
    float s = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[k][i][j] = raw_at(raw[k][i], j);
        s += v[k][i][j];
      }
    const float mean = row_sum<G>(s, sm[0][k]) / (float)N;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if ((i * G + t) * VEC < N) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[k][i][j] -= mean;
          q += v[k][i][j] * v[k][i][j];
        }
      }
    rstd[k] = 1.0f / sqrtf(row_sum<G>(q, sm[1][k]) / (float)N + eps);
    if (t == 0 && (RP == 1 || row0 + k < M)) {
      if (mean_out) mean_out[row0 + k] = mean;
      if (rstd_out) rstd_out[row0 + k] = rstd[k];
    }
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (i * G + t) * VEC;
    if (c < N) {
      float gm[VEC], bt[VEC], o[VEC];
      if (gamma) load_vec<WT, VEC>(gamma + c, gm);
      if (beta) load_vec<WT, VEC>(beta + c, bt);
#pragma unroll
      for (int k = 0; k < RP; ++k) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = v[k][i][j] * rstd[k];
          o[j] = (gamma ? h * gm[j] : h) + (beta ? bt[j] : 0.f);
        }
        if (RP == 1 || row0 + k < M) store_vec<XT, VEC>(y + (row0 + k) * ldy + c, o);
      }
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
  __shared__ float sm[2][32];
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const XT* xr = x + row * ldx;
    float s = 0.f, q = 0.f;
    for (int64_t c = threadIdx.x; c < N; c += 1024) s += to_f(xr[c]);
    const float mean = row_sum<1024>(s, sm[0]) / (float)N;
    for (int64_t c = threadIdx.x; c < N; c += 1024) {
      const float d = to_f(xr[c]) - mean;
      q += d * d;
    }
    const float rstd = 1.0f / sqrtf(row_sum<1024>(q, sm[1]) / (float)N + eps);
    if (threadIdx.x == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
    for (int64_t c = threadIdx.x; c < N; c += 1024) {
      const float h = (to_f(xr[c]) - mean) * rstd;
      const float o = (gamma ? h * to_f(gamma[c]) : h) + (beta ? to_f(beta[c]) : 0.f);
      y[row * ldy + c] = from_f<XT>(o);
    }
  }
}

// Backward. A group of G threads (a warp of eight in a block, or a whole block) walks rows; a
// thread owns the same PER * VEC columns of every row and keeps their dgamma and dbeta sums in
// registers until the end. Each thread copies its own columns of the next S - 1 rows into a ring
// in shared memory (cp.async), so that 64 to 190 KB are on their way on an SM and no barrier is
// spent on the copies; VEC = 1 (rows off 16-byte boundaries) loads directly.
template <typename XT, int VEC, int B, int PER, int S>
constexpr int ring_bytes() {
  return VEC > 1 ? S * PER * 2 * B * 16 : 0;
}
MOE_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <typename XT, typename WT, int VEC, int G, int PER, int S>
__global__ void __launch_bounds__(G < 256 ? 256 : G) ln_bwd_kernel(
    const XT* dy, int64_t lddy, const XT* x, int64_t ldx, const WT* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, XT* dx, int64_t lddx,
    float* __restrict__ part, WT* __restrict__ dgamma, WT* __restrict__ dbeta, int64_t M,
    int N) {
  MOE_GRIDDEP_ENTRY();
  constexpr int B = G < 256 ? 256 : G, GROUPS = B / G;
  constexpr bool kRing = VEC > 1;
  // few enough columns a thread to hold gamma and one row's widened values beside the sums
  constexpr bool kKeep = PER * VEC <= 16 && G <= 512;
  __shared__ float sm[2][2][32];
  extern __shared__ uint4 ring[];  // [S][2 PER][B]
  const int t = threadIdx.x % G;
  const int64_t row0 = (int64_t)blockIdx.x * GROUPS + threadIdx.x / G;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const uint32_t ring0 = smem_u32(ring) + threadIdx.x * 16;
  auto fetch = [&](int64_t row, int slot) {
    if (row < M) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = (i * G + t) * VEC;
        if (c < N) {
          cp_async16(ring0 + ((slot * 2 * PER + 2 * i) * B) * 16, x + row * ldx + c);
          cp_async16(ring0 + ((slot * 2 * PER + 2 * i + 1) * B) * 16, dy + row * lddy + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto ring_at = [&](int slot, int i) {
    const uint4 q = ring[(slot * 2 * PER + i) * B + threadIdx.x];
    Raw<XT, VEC> r;
    r.w[0] = q.x;
    if constexpr (VEC > 1) {
      r.w[1] = q.y;
      r.w[2] = q.z;
      r.w[3] = q.w;
    }
    return r;
  };
  float dg[PER][VEC], db[PER][VEC];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;
  if constexpr (kRing) {
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch(row0 + k * step, k);
  }
  float gm[kKeep ? PER : 1][VEC];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) gm[i][j] = 1.0f;
      if (gamma && c < N) load_vec<WT, VEC>(gamma + c, gm[i]);
    }
  }
  int slot = 0, turn = 0;
  float mu = row0 < M ? mean[row0] : 0.f, rs = row0 < M ? rstd[row0] : 0.f;
  for (int64_t row = row0; row < M; row += step) {
    Raw<XT, VEC> h[PER], u[PER];
    if constexpr (kRing) {
      const int ahead = slot == 0 ? S - 1 : slot - 1;
      fetch(row + (S - 1) * step, ahead);
      asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        h[i] = ring_at(slot, 2 * i);
        u[i] = ring_at(slot, 2 * i + 1);
      }
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = (i * G + t) * VEC;
        if (c < N) {
          load_raw(x + row * ldx + c, h[i]);
          load_raw(dy + row * lddy + c, u[i]);
        }
      }
    }
    const float m0 = mu, r0 = rs;
    if (row + step < M) {  // the next row's statistics
      mu = mean[row + step];
      rs = rstd[row + step];
    }
    // c = x - mean; the sums over the row are of u and u c, rstd goes into their factors
    float c_[kKeep ? PER : 1][VEC], u_[kKeep ? PER : 1][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC;
      if (c < N) {
        float gv[VEC];
        if (!kKeep && gamma) load_vec<WT, VEC>(gamma + c, gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float cj = raw_at(h[i], j) - m0, d = raw_at(u[i], j);
          dg[i][j] += (d * r0) * cj;
          db[i][j] += d;
          const float uj = kKeep ? d * gm[kKeep ? i : 0][j] : gamma ? d * gv[j] : d;
          s1 += uj;
          s2 += uj * cj;
          if (kKeep) {
            c_[kKeep ? i : 0][j] = cj;
            u_[kKeep ? i : 0][j] = uj;
          }
        }
      }
    }
    row_sum2<G>(s1, s2, sm, turn);
    turn ^= 1;
    const float k1 = r0 * (s1 / (float)N), k2 = (r0 * r0) * r0 * (s2 / (float)N);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC;
      if (c < N) {
        if constexpr (!kKeep && kRing) {  // once more from the ring: registers are short here
          h[i] = ring_at(slot, 2 * i);
          u[i] = ring_at(slot, 2 * i + 1);
        }
        float gv[VEC], o[VEC];
        if (!kKeep && gamma) load_vec<WT, VEC>(gamma + c, gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float cj, uj;
          if constexpr (kKeep) {
            cj = c_[i][j];
            uj = u_[i][j];
          } else {
            const float d = raw_at(u[i], j);
            cj = raw_at(h[i], j) - m0;
            uj = gamma ? d * gv[j] : d;
          }
          o[j] = (r0 * uj - k1) - cj * k2;
        }
        store_vec<XT, VEC>(dx + row * lddx + c, o);
      }
    }
    if (kRing && ++slot == S) slot = 0;
  }
  if (!part) return;
  float* pg = part + (int64_t)blockIdx.x * 2 * N;  // a single block writes the results
  if constexpr (kRing) asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (GROUPS > 1) {
    // the block's groups, in order, through the columns of one shared row at a time
    __shared__ float cols[2][G * PER * VEC];
    for (int g = 0; g < GROUPS; ++g) {
      __syncthreads();
      if ((int)threadIdx.x / G == g) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            const int c = (i * G + t) * VEC + j;
            cols[0][c] = g == 0 ? dg[i][j] : cols[0][c] + dg[i][j];
            cols[1][c] = g == 0 ? db[i][j] : cols[1][c] + db[i][j];
          }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < N; c += B) {
      if (gridDim.x == 1) {
        if (dgamma) dgamma[c] = from_f<WT>(cols[0][c]);
        if (dbeta) dbeta[c] = from_f<WT>(cols[1][c]);
      } else {
        pg[c] = cols[0][c];
        pg[N + c] = cols[1][c];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC;
      if (c < N) {
        if (gridDim.x == 1) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) {
            if (dgamma) dgamma[c + j] = from_f<WT>(dg[i][j]);
            if (dbeta) dbeta[c + j] = from_f<WT>(db[i][j]);
          }
        } else if constexpr (VEC > 1) {  // N is a multiple of VEC, the partials 16-byte aligned
#pragma unroll
          for (int j = 0; j < VEC; j += 4) {
            *reinterpret_cast<float4*>(pg + c + j) =
                make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
            *reinterpret_cast<float4*>(pg + N + c + j) =
                make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
          }
        } else {
          pg[c] = dg[i][0];
          pg[N + c] = db[i][0];
        }
      }
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
  __shared__ float sm[2][2][32];
  int turn = 0;
  for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
    const float mu = mean[row], rs = rstd[row];
    float s1 = 0.f, s2 = 0.f;
    for (int64_t c = threadIdx.x; c < N; c += 1024) {
      const float d = to_f(dy[row * lddy + c]);
      const float u = gamma ? d * to_f(gamma[c]) : d;
      s1 += u;
      s2 += u * ((to_f(x[row * ldx + c]) - mu) * rs);
    }
    row_sum2<1024>(s1, s2, sm, turn);
    turn ^= 1;
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

// dgamma[c] (columns [0, N)) and dbeta (columns [N, 2N)) = sum of the blocks' partials. Each of a
// block's 32 warps sums every 32nd partial of 32 columns; the warps' sums are added in order.
template <typename WT>
__global__ void __launch_bounds__(1024) ln_colsum_kernel(const float* __restrict__ part,
                                                         int nparts, int64_t N,
                                                         WT* __restrict__ dgamma,
                                                         WT* __restrict__ dbeta) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * N) {
#pragma unroll 5
    for (int b = w; b < nparts; b += 32) s += part[(int64_t)b * 2 * N + c];
  }
  sm[w][lane] = s;
  __syncthreads();
  // warp w holds column w's 32 sums: lane l that of warp l
  s = sm[lane][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int64_t col = (int64_t)blockIdx.x * 32 + w;
  if (lane == 0 && col < 2 * N) {
    if (col < N) {
      if (dgamma) dgamma[col] = from_f<WT>(s);
    } else if (dbeta) {
      dbeta[col - N] = from_f<WT>(s);
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
  void *dgamma, *dbeta;
  float* part;
  int nparts;
  bool done;  // the weight gradients are final
  cudaStream_t s;
};

template <typename XT, typename WT, int VEC, int G, int PER, int RP = 1>
cudaError_t fwd_launch(const LnArgs& a) {
  constexpr int B = G < 128 ? 128 : G, rows = B / G * RP;
  const int64_t blocks = (a.M + rows - 1) / rows;
  return launch_pdl(ln_fwd_kernel<XT, WT, VEC, G, PER, RP>, (unsigned)blocks, B, 0, a.s, 1,
                    static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma),
                    static_cast<const WT*>(a.beta), static_cast<XT*>(a.y), a.ldy, a.mean, a.rstd,
                    a.M, (int)a.N, a.eps);
}

template <typename XT, typename WT>
cudaError_t fwd_typed(const LnArgs& a) {
  constexpr int V = 16 / sizeof(XT);
  // Weights wider than the rows cost more L1 reads than the rows: two rows share them (16384 x
  // 2880 bf16 rows, fp32 weights: 35.4 us against 42.7). With equal types the registers of a
  // second row cost more than it saves (8192 x 4096 bf16: 29.8 us against 23.2).
  constexpr int RP = sizeof(WT) > sizeof(XT) ? 2 : 1;
  const bool vec = a.N % V == 0 && a.ldx % V == 0 && a.ldy % V == 0 && aligned_to(a.x, 16) &&
                   aligned_to(a.y, 16) && aligned_to(a.gamma, 16) && aligned_to(a.beta, 16);
  const int64_t N = a.N;
  // Up to 32 elements a thread: as few warps a row as hold it, for many rows in flight; with too
  // few rows to fill the GPU that way, as many threads as the row feeds, which is there sooner.
  const bool many = a.M >= (int64_t)std::max(device_sms(), 1) * 2;
  if (vec) {
    constexpr int P = 32 / V;  // vectors of 32 elements
    if (N <= 32 * V) return fwd_launch<XT, WT, V, 32, 1>(a);
    if (many) {
      if (N <= 32 * 2 * V) return fwd_launch<XT, WT, V, 32, 2>(a);
      if (N <= 32 * 32) return fwd_launch<XT, WT, V, 32, P>(a);
      if (N <= 128 * 16) return fwd_launch<XT, WT, V, 128, P / 2, RP>(a);
      if (N <= 128 * 24) return fwd_launch<XT, WT, V, 128, P / 4 * 3, RP>(a);
      if (N <= 128 * 32) return fwd_launch<XT, WT, V, 128, P, RP>(a);
      if (N <= 256 * 32) return fwd_launch<XT, WT, V, 256, P, RP>(a);
      if (N <= 512 * 32) return fwd_launch<XT, WT, V, 512, P, RP>(a);
    }
    if (N <= 256 * V) return fwd_launch<XT, WT, V, 256, 1>(a);
    if (N <= 512 * V) return fwd_launch<XT, WT, V, 512, 1>(a);
    if (N <= 1024 * V) return fwd_launch<XT, WT, V, 1024, 1>(a);
    if (N <= 1024 * 16) return fwd_launch<XT, WT, V, 1024, 16 / V>(a);
    if (N <= 1024 * 32) return fwd_launch<XT, WT, V, 1024, P>(a);
  } else {
    if (N <= 32 * 8) return fwd_launch<XT, WT, 1, 32, 8>(a);
    if (many) {
      if (N <= 32 * 16) return fwd_launch<XT, WT, 1, 32, 16>(a);
      if (N <= 32 * 32) return fwd_launch<XT, WT, 1, 32, 32>(a);
      if (N <= 128 * 24) return fwd_launch<XT, WT, 1, 128, 24>(a);
    }
    if (N <= 1024 * 4) return fwd_launch<XT, WT, 1, 1024, 4>(a);
    if (N <= 1024 * 16) return fwd_launch<XT, WT, 1, 1024, 16>(a);
  }
  const int grid = (int)std::min<int64_t>(a.M, (int64_t)std::max(device_sms(), 1) * 2);
  return launch_pdl(ln_fwd_long_kernel<XT, WT>, grid, 1024, 0, a.s, 1,
                    static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma),
                    static_cast<const WT*>(a.beta), static_cast<XT*>(a.y), a.ldy, a.mean, a.rstd,
                    a.M, a.N, a.eps);
}

template <typename XT, typename WT, int VEC, int G, int PER, int S>
cudaError_t bwd_launch(LnArgs& a) {
  constexpr int B = G < 256 ? 256 : G, GROUPS = B / G;
  constexpr int smem = ring_bytes<XT, VEC, B, PER, S>();
  auto kern = ln_bwd_kernel<XT, WT, VEC, G, PER, S>;
  if (smem > 0) {
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
    if (e != cudaSuccess) return e;
  }
  // as many blocks as fit at once (at least two where registers allow), each a row of partials
  static const int per_sm = [&] {
    int n = 0;
    return cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, B, smem) == cudaSuccess && n > 0
               ? n : 1;
  }();
  const int64_t fit = (int64_t)std::max(device_sms(), 1) * per_sm;
  a.nparts = (int)std::max<int64_t>(
      1, std::min<int64_t>((a.M + GROUPS - 1) / GROUPS, std::min<int64_t>(fit, max_parts(a.N))));
  a.done = a.nparts == 1;
  return launch_pdl(kern, a.nparts, B, smem, a.s, 1, static_cast<const XT*>(a.dy), a.lddy,
                    static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma), a.mean,
                    a.rstd, static_cast<XT*>(a.dx), a.lddx, a.part, static_cast<WT*>(a.dgamma),
                    static_cast<WT*>(a.dbeta), a.M, (int)a.N);
}

template <typename XT, typename WT>
cudaError_t bwd_typed(LnArgs& a) {
  constexpr int V = 16 / sizeof(XT);
  const bool vec = a.N % V == 0 && a.ldx % V == 0 && a.lddy % V == 0 && a.lddx % V == 0 &&
                   aligned_to(a.x, 16) && aligned_to(a.dy, 16) && aligned_to(a.dx, 16) &&
                   aligned_to(a.gamma, 16);
  const int64_t N = a.N;
  if (vec) {
    if (N <= 32 * V) return bwd_launch<XT, WT, V, 32, 1, 4>(a);
    if (N <= 32 * 2 * V) return bwd_launch<XT, WT, V, 32, 2, 3>(a);
    if (N <= 32 * 4 * V) return bwd_launch<XT, WT, V, 32, 4, 3>(a);
    if (N <= 256 * V) return bwd_launch<XT, WT, V, 256, 1, 4>(a);
    if (N <= 256 * 2 * V) return bwd_launch<XT, WT, V, 256, 2, 4>(a);
    if constexpr (sizeof(XT) == 4) {
      if (N <= 256 * 4 * V) return bwd_launch<XT, WT, V, 256, 4, 3>(a);
    } else {
      if (N <= 512 * 2 * V) return bwd_launch<XT, WT, V, 512, 2, 3>(a);
    }
    if (N <= 512 * 4 * V) return bwd_launch<XT, WT, V, 512, 4, 3>(a);
    if constexpr (sizeof(XT) == 4)
      if (N <= 512 * 8 * V) return bwd_launch<XT, WT, V, 512, 8, 1>(a);
  } else {
    if (N <= 32 * 8) return bwd_launch<XT, WT, 1, 32, 8, 1>(a);
    if (N <= 256 * 4) return bwd_launch<XT, WT, 1, 256, 4, 1>(a);
    if (N <= 512 * 8) return bwd_launch<XT, WT, 1, 512, 8, 1>(a);
    if (N <= 512 * 32) return bwd_launch<XT, WT, 1, 512, 32, 1>(a);
  }
  const int64_t most = std::min<int64_t>(std::max(device_sms(), 1), max_parts(N));
  a.nparts = (int)std::min<int64_t>(a.M, most);
  if (a.part) {
    cudaError_t e = launch_pdl(ln_bwd_cols_long_kernel<XT>, a.nparts, 256, 0, a.s, 1,
                               static_cast<const XT*>(a.dy), a.lddy, static_cast<const XT*>(a.x),
                               a.ldx, a.mean, a.rstd, a.part, a.M, a.N);
    count_launch(a.s, MOE_K_LAYERNORM_BWD);
    if (e != cudaSuccess) return e;
  }
  const int grid = (int)std::min<int64_t>(a.M, (int64_t)std::max(device_sms(), 1) * 2);
  return launch_pdl(ln_bwd_rows_long_kernel<XT, WT>, grid, 1024, 0, a.s, 1,
                    static_cast<const XT*>(a.dy), a.lddy, static_cast<const XT*>(a.x), a.ldx,
                    static_cast<const WT*>(a.gamma), a.mean, a.rstd, static_cast<XT*>(a.dx),
                    a.lddx, a.M, a.N);
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
  cudaError_t e = x_dtype == MOE_DT_FP32   ? fwd_typed<float, float>(a)
                  : w_dtype == MOE_DT_FP32 ? fwd_typed<__nv_bfloat16, float>(a)
                                           : fwd_typed<__nv_bfloat16, __nv_bfloat16>(a);
  count_launch(a.s, MOE_K_LAYERNORM_FWD);
  if (e != cudaSuccess) return cuda_fail(e, "layernorm forward launch");
  return MOE_OK;
}

size_t moe_layernorm_workspace(int64_t M, int64_t N) {
  if (M < 0 || N < 1 || M > INT32_MAX || N > INT32_MAX) {
    fail(MOE_ERR_INVALID_ARG, "M must be in [0, 2^31) and N in [1, 2^31)");
    return 0;
  }
  return (size_t)std::max<int64_t>(1, std::min<int64_t>(M, max_parts(N))) * 2 * N * sizeof(float);
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
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (M > 0) {
    e = x_dtype == MOE_DT_FP32   ? bwd_typed<float, float>(a)
        : w_dtype == MOE_DT_FP32 ? bwd_typed<__nv_bfloat16, float>(a)
                                 : bwd_typed<__nv_bfloat16, __nv_bfloat16>(a);
    count_launch(a.s, MOE_K_LAYERNORM_BWD);
    if (e != cudaSuccess) return cuda_fail(e, "layernorm backward launch");
  }  // no rows: no partials, the sums are zero
  if (weights && !a.done) {
    const unsigned grid = (unsigned)((2 * N + 31) / 32);
    if (w_dtype == MOE_DT_FP32)
      e = launch_pdl(ln_colsum_kernel<float>, grid, 1024, 0, a.s, 1, (const float*)a.part,
                         a.nparts, N, static_cast<float*>(dgamma), static_cast<float*>(dbeta));
    else
      e = launch_pdl(ln_colsum_kernel<__nv_bfloat16>, grid, 1024, 0, a.s, 1,
                         (const float*)a.part, a.nparts, N, static_cast<__nv_bfloat16*>(dgamma),
                         static_cast<__nv_bfloat16*>(dbeta));
    count_launch(a.s, MOE_K_LAYERNORM_REDUCE);
    if (e != cudaSuccess) return cuda_fail(e, "layernorm reduction launch");
  }
  return MOE_OK;
}

}  // extern "C"
