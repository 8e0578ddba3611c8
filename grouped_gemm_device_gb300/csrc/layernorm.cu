// Layer norm over the last dimension, forward and backward (moe_layernorm_fwd /
// moe_layernorm_bwd in include/moegmm.h).
//
//   y = (x - mean) rstd gamma + beta;  h = (x - mean) rstd, u = dy gamma:
//   dx = rstd (u - mean_n(u) - h mean_n(u h));  dgamma = sum_m dy h;  dbeta = sum_m dy
//
// Bound by HBM: the forward reads and writes M N elements once, the backward reads x and dy and
// writes dx once. A row stays in registers between its statistics and its use, so the variance is
// taken about the mean (two passes over registers, not E[x^2] - mean^2). Statistics, sums and the
// weight-gradient partials are fp32. With inputs from HBM: forward of 8192 x 4096 bf16 23 us (5.7
// TB/s), of 16384 x 2880 with fp32 weights 35 us (5.3 TB/s), of 4096 x 7168 fp32 38 us (6.2 TB/s),
// of one row of 7168 2.1 us; backward of 8192 x 4096 bf16 42 us (4.8 TB/s), of 4096 x 7168 fp32 59
// us (5.9 TB/s), of which the sum of the partials takes about 4. Widening bf16 runs at half the rate of the products, so it
// is done once a value where the registers allow.
#include "kernels.cuh"
#include "realign.cuh"

namespace moe {
namespace {

// Backward blocks at most (rows of the partial weight gradients), by the row's length: short rows
// leave small partials and run more blocks.
constexpr int64_t kShortRow = 1024;
int64_t max_parts(int64_t N) { return N <= kShortRow ? 960 : 480; }
// A row of partials: two of this many floats, whole vectors of any type and the place of a row's
// first element in its first block.
template <typename I>
__host__ __device__ I pad_cols(I N) {
  return (N + 7) / 8 * 8 + 8;
}

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

// VEC consecutive elements as they lie in memory: 16 bytes.
template <typename T, int VEC>
struct Raw {
  uint32_t w[4];
  static_assert(VEC * sizeof(T) == 16, "16 bytes");
};
template <typename T, int VEC>
MOE_DEVICE void zero_raw(Raw<T, VEC>& r) {
#pragma unroll
  for (uint32_t& w : r.w) w = 0u;
}
// Streamed data is not kept in L1, which the weights of the following rows want.
template <typename T, int VEC>
MOE_DEVICE void load_raw(const T* p, Raw<T, VEC>& r) {
  asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3])
               : "l"(p));
}
// Zeros before element lo and from element hi on.
template <typename T, int VEC>
MOE_DEVICE void clear_outside(Raw<T, VEC>& r, int lo, int hi) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) {
      if (k < lo || k >= hi) r.w[k] = 0u;
    } else {
      if (2 * k < lo || 2 * k >= hi) r.w[k] &= 0xFFFF0000u;
      if (2 * k + 1 < lo || 2 * k + 1 >= hi) r.w[k] &= 0x0000FFFFu;
    }
  }
}
template <typename T, int VEC>
MOE_DEVICE float raw_at(const Raw<T, VEC>& r, int j) {  // j is a constant after unrolling
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[j]);
  else return (j & 1) ? bf16_hi(r.w[j >> 1]) : bf16_lo(r.w[j >> 1]);
}

// VEC consecutive elements (VEC * sizeof(T) a multiple of 16 bytes) as fp32.
template <typename T, int VEC>
MOE_DEVICE void load_vec(const T* p, float (&v)[VEC]) {
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
// The weights of columns c .. c + VEC - 1. ANY: c may be any column from 1 - VEC on (zeros outside
// [0, N)), and (vec false) p off a 16-byte boundary.
template <bool ANY, typename T, int VEC>
MOE_DEVICE void load_weights(const T* p, int c, int N, bool vec, float (&v)[VEC]) {
  if constexpr (!ANY) {
    load_vec<T, VEC>(p + c, v);
  } else if (vec) {
    constexpr int E = 16 / sizeof(T), W = VEC / E;  // elements of 16 bytes, such blocks to fill
    const int b = (c + VEC) / E - W;                // the block of c, rounded down
    uint32_t w[4 * W + 4];
#pragma unroll
    for (int i = 0; i <= W; ++i) {
      uint4 q = make_uint4(0, 0, 0, 0);
      if (b + i >= 0 && (b + i) * E < N) q = __ldg(reinterpret_cast<const uint4*>(p) + b + i);
      w[4 * i] = q.x;
      w[4 * i + 1] = q.y;
      w[4 * i + 2] = q.z;
      w[4 * i + 3] = q.w;
    }
    drop_bytes(w, (c - b * E) * (int)sizeof(T));
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      if constexpr (sizeof(T) == 4) v[j] = __uint_as_float(w[j]);
      else v[j] = (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
    }
    if (c < 0 || c + VEC > N) {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c + j < 0 || c + j >= N) v[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = c + j >= 0 && c + j < N ? to_f(__ldg(p + c + j)) : 0.f;
  }
}
template <typename T, int VEC>
MOE_DEVICE void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                   pack_bf16x2(v[6], v[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
}
// The same of the elements [lo, hi).
template <typename T, int VEC>
MOE_DEVICE void store_part(T* p, const float (&v)[VEC], int lo, int hi) {
#pragma unroll
  for (int j = 0; j < VEC; ++j)
    if (j >= lo && j < hi) p[j] = from_f<T>(v[j]);
}
// Rows off 16-byte boundaries (ANY): a thread owns whole aligned blocks of 16 bytes, so that rows
// are read and written like aligned ones. Element j of block b is then column b VEC - lead + j,
// `lead` the row's first element's place in its first block; every kCycle-th row has the same one,
// and a thread takes only rows that agree. What a row's first and last block hold of the rows
// beside it is cleared when read and left alone when written. (Moving the bytes between columns
// and blocks for every row instead: 8192 x 4095 bf16, 52 us forward and 88 us backward.)
constexpr int kCycle = 8;
template <typename T>
MOE_DEVICE int row_lead(const T* row) {
  return lead_bytes(row) / (int)sizeof(T);
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
// a thread and row: N <= G * PER * VEC (ANY: N + VEC - 1). The rows share each load of the weights.
// Six blocks an SM where the registers allow (16384 x 2880, fp32 weights: 35 us; with five 44).
template <typename XT, typename WT, int VEC, int G, int PER, int RP, bool ANY>
__global__ void __launch_bounds__(G < 128 ? 128 : G, G <= 128 && PER * VEC * RP <= 48 ? 6 : 1)
    ln_fwd_kernel(
    const XT* x, int64_t ldx, const WT* __restrict__ gamma, const WT* __restrict__ beta, XT* y,
    int64_t ldy, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t M, int N,
    float eps, int wvec) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[2][RP][32];
  constexpr int R = (G < 128 ? 128 : G) / G;  // groups a block
  static_assert(!ANY || RP == 1, "rows beside one another lie differently in their blocks");
  const int t = threadIdx.x % G;
  const int64_t g = (int64_t)blockIdx.x * R + threadIdx.x / G;
  const int64_t row0 = g * RP;
  if (G == 32 && row0 >= M) return;  // a block's groups are its warps; otherwise R = 1
  const int lead = ANY ? row_lead(x + row0 * ldx) : 0;
  Raw<XT, VEC> raw[RP][PER];
#pragma unroll
  for (int k = 0; k < RP; ++k)
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      zero_raw(raw[k][i]);
      if (c < N && (RP == 1 || row0 + k < M)) {
        load_raw(x + (row0 + k) * ldx + c, raw[k][i]);
        if (ANY && (c < 0 || c + VEC > N)) clear_outside(raw[k][i], -c, N - c);
      }
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
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      if (c < N) {
        if (ANY && (c < 0 || c + VEC > N)) {  // nothing from outside the row
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (c + j < 0 || c + j >= N) v[k][i][j] = mean;
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[k][i][j] -= mean;
          q += v[k][i][j] * v[k][i][j];
        }
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
    const int c = (i * G + t) * VEC - lead;
    if (c < N) {
      float gm[VEC], bt[VEC], o[VEC];
      if (gamma) load_weights<ANY, WT, VEC>(gamma, c, N, wvec, gm);
      if (beta) load_weights<ANY, WT, VEC>(beta, c, N, wvec, bt);
#pragma unroll
      for (int k = 0; k < RP; ++k) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = v[k][i][j] * rstd[k];
          o[j] = (gamma ? h * gm[j] : h) + (beta ? bt[j] : 0.f);
        }
        if (RP == 1 || row0 + k < M) {
          XT* at = y + (row0 + k) * ldy + c;
          if (!ANY || (c >= 0 && c + VEC <= N)) store_vec<XT, VEC>(at, o);
          else store_part<XT, VEC>(at, o, -c, N - c);
        }
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

// Threads a block of the kernels that walk rows: eight warps with a row each, or one row.
constexpr int block_of(int G) { return G == 32 ? 256 : G; }
template <int N>
MOE_DEVICE void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
MOE_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Many rows off 16-byte boundaries: a group of G threads (a warp of eight in a block, or a whole
// block) walks rows that lie alike in their blocks, with the weights of its columns in registers
// and the next S - 1 rows on their way to shared memory (cp.async, a thread's own columns).
// N + VEC - 1 <= G * PER * VEC.
template <typename XT, typename WT, int VEC, int G, int PER, int S>
__global__ void __launch_bounds__(block_of(G)) ln_fwd_walk_kernel(
    const XT* x, int64_t ldx, const WT* __restrict__ gamma, const WT* __restrict__ beta, XT* y,
    int64_t ldy, float* __restrict__ mean_out, float* __restrict__ rstd_out, int64_t M, int N,
    float eps, int wvec) {
  MOE_GRIDDEP_ENTRY();
  constexpr int B = block_of(G), GROUPS = B / G;
  __shared__ float sm[2][2][32];
  extern __shared__ uint4 ring[];  // [S][PER][B]
  const int t = threadIdx.x % G;
  const int64_t row0 = (int64_t)blockIdx.x * GROUPS + threadIdx.x / G;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const uint32_t ring0 = smem_u32(ring) + threadIdx.x * 16;
  const int lead = row_lead(x + row0 * ldx);
  auto fetch = [&](int64_t row, int slot) {
    if (row < M) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = (i * G + t) * VEC - lead;
        if (c < N) cp_async16(ring0 + ((slot * PER + i) * B) * 16, x + row * ldx + c);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch(row0 + k * step, k);
  float gm[PER][VEC], bt[PER][VEC];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (i * G + t) * VEC - lead;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      gm[i][j] = 1.0f;
      bt[i][j] = 0.f;
    }
    if (gamma && c < N) load_weights<true, WT, VEC>(gamma, c, N, wvec, gm[i]);
    if (beta && c < N) load_weights<true, WT, VEC>(beta, c, N, wvec, bt[i]);
  }
  int slot = 0, turn = 0;
  for (int64_t row = row0; row < M; row += step) {
    fetch(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    float v[PER][VEC], s = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      const uint4 w = ring[(slot * PER + i) * B + threadIdx.x];
      Raw<XT, VEC> r;
      r.w[0] = w.x;
      r.w[1] = w.y;
      r.w[2] = w.z;
      r.w[3] = w.w;
      if (c < 0 || c + VEC > N) clear_outside(r, -c, N - c);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] = raw_at(r, j);
        s += v[i][j];
      }
    }
    const float mean = row_sum<G>(s, sm[turn][0]) / (float)N;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      if (c < 0 || c + VEC > N) {  // nothing from outside the row
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < 0 || c + j >= N) v[i][j] = mean;
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        v[i][j] -= mean;
        q += v[i][j] * v[i][j];
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<G>(q, sm[turn][1]) / (float)N + eps);
    turn ^= 1;
    if (t == 0) {
      if (mean_out) mean_out[row] = mean;
      if (rstd_out) rstd_out[row] = rstd;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      if (c < N) {
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float h = v[i][j] * rstd;
          o[j] = (gamma ? h * gm[i][j] : h) + bt[i][j];
        }
        XT* at = y + row * ldy + c;
        if (c >= 0 && c + VEC <= N) store_vec<XT, VEC>(at, o);
        else store_part<XT, VEC>(at, o, -c, N - c);
      }
    }
    if (++slot == S) slot = 0;
  }
  cp_async_wait<0>();
}

// Backward. A group of G threads (a warp of eight in a block, or a whole block) walks rows; a
// thread owns the same PER * VEC columns of every row and keeps their dgamma and dbeta sums in
// registers until the end. Each thread copies its own columns of the next S - 1 rows into a ring
// in shared memory (cp.async), so that 64 to 190 KB are on their way on an SM and no barrier is
// spent on the copies. ANY: N + VEC - 1 <= G * PER * VEC, and the groups' number a multiple of
// kCycle where a group takes more than one row.
template <int B, int PER, int S>
constexpr int ring_bytes() {
  return S * PER * 2 * B * 16;
}
template <typename XT, typename WT, int VEC, int G, int PER, int S, bool ANY>
__global__ void __launch_bounds__(block_of(G)) ln_bwd_kernel(
    const XT* dy, int64_t lddy, const XT* x, int64_t ldx, const WT* __restrict__ gamma,
    const float* __restrict__ mean, const float* __restrict__ rstd, XT* dx, int64_t lddx,
    float* __restrict__ part, WT* __restrict__ dgamma, WT* __restrict__ dbeta, int64_t M,
    int N, int wvec) {
  MOE_GRIDDEP_ENTRY();
  constexpr int B = block_of(G), GROUPS = B / G;
  // few enough columns a thread to hold gamma and one row's widened values beside the sums
  constexpr bool kKeep = PER * VEC <= 16 && G <= 512;
  __shared__ float sm[2][2][32];
  extern __shared__ uint4 ring[];  // [S][2 PER][B]
  const int t = threadIdx.x % G;
  const int64_t row0 = (int64_t)blockIdx.x * GROUPS + threadIdx.x / G;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const uint32_t ring0 = smem_u32(ring) + threadIdx.x * 16;
  const int lead = ANY ? row_lead(x + row0 * ldx) : 0;
  auto fetch = [&](int64_t row, int slot) {
    if (row < M) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = (i * G + t) * VEC - lead;
        if (c < N) {
          cp_async16(ring0 + ((slot * 2 * PER + 2 * i) * B) * 16, x + row * ldx + c);
          cp_async16(ring0 + ((slot * 2 * PER + 2 * i + 1) * B) * 16, dy + row * lddy + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto ring_at = [&](int slot, int i, int which) {  // vector i of a row's x (0) or dy (1)
    const uint4 q = ring[(slot * 2 * PER + 2 * i + which) * B + threadIdx.x];
    Raw<XT, VEC> r;
    r.w[0] = q.x;
    r.w[1] = q.y;
    r.w[2] = q.z;
    r.w[3] = q.w;
    const int c = (i * G + t) * VEC - lead;
    if (ANY && (c < 0 || c + VEC > N)) clear_outside(r, -c, N - c);
    return r;
  };
  float dg[PER][VEC], db[PER][VEC];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[i][j] = db[i][j] = 0.f;
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch(row0 + k * step, k);
  float gm[kKeep ? PER : 1][VEC];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
#pragma unroll
      for (int j = 0; j < VEC; ++j) gm[i][j] = 1.0f;
      if (gamma && c < N) load_weights<ANY, WT, VEC>(gamma, c, N, wvec, gm[i]);
    }
  }
  int slot = 0, turn = 0;
  float mu = row0 < M ? mean[row0] : 0.f, rs = row0 < M ? rstd[row0] : 0.f;
  for (int64_t row = row0; row < M; row += step) {
    Raw<XT, VEC> xv[PER], dv[PER];
    const int ahead = slot == 0 ? S - 1 : slot - 1;
    fetch(row + (S - 1) * step, ahead);
    cp_async_wait<S - 1>();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      xv[i] = ring_at(slot, i, 0);
      dv[i] = ring_at(slot, i, 1);
    }
    const float m0 = mu, r0 = rs;
    if (row + step < M) {  // the next row's statistics
      mu = mean[row + step];
      rs = rstd[row + step];
    }
    // h = (x - mean) rstd is formed first: products of rstd alone leave fp32's range (rstd^3 is 0
    // for rows of a spread above 1e15) where h, u and dx do not
    float h_[kKeep ? PER : 1][VEC], u_[kKeep ? PER : 1][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      if (c < N) {
        float gv[VEC];
        if (!kKeep && gamma) load_weights<ANY, WT, VEC>(gamma, c, N, wvec, gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float hj = (raw_at(xv[i], j) - m0) * r0, d = raw_at(dv[i], j);
          dg[i][j] += d * hj;
          db[i][j] += d;
          const float uj = kKeep ? d * gm[kKeep ? i : 0][j] : gamma ? d * gv[j] : d;
          s1 += uj;
          s2 += uj * hj;
          if (kKeep) {
            h_[kKeep ? i : 0][j] = hj;
            u_[kKeep ? i : 0][j] = uj;
          }
        }
      }
    }
    row_sum2<G>(s1, s2, sm, turn);
    turn ^= 1;
    const float k1 = r0 * (s1 / (float)N), k2 = r0 * (s2 / (float)N);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      if (c < N) {
        if (!kKeep) {  // once more from the ring: registers are short here
          xv[i] = ring_at(slot, i, 0);
          dv[i] = ring_at(slot, i, 1);
        }
        float gv[VEC], o[VEC];
        if (!kKeep && gamma) load_weights<ANY, WT, VEC>(gamma, c, N, wvec, gv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float hj, uj;
          if constexpr (kKeep) {
            hj = h_[i][j];
            uj = u_[i][j];
          } else {
            const float d = raw_at(dv[i], j);
            hj = (raw_at(xv[i], j) - m0) * r0;
            uj = gamma ? d * gv[j] : d;
          }
          o[j] = (r0 * uj - k1) - hj * k2;
        }
        XT* at = dx + row * lddx + c;
        if (!ANY || (c >= 0 && c + VEC <= N)) store_vec<XT, VEC>(at, o);
        else store_part<XT, VEC>(at, o, -c, N - c);
      }
    }
    if (++slot == S) slot = 0;
  }
  if (!part) return;
  const int NP = pad_cols(N);
  float* pg = part + (int64_t)blockIdx.x * 2 * NP;  // a single block writes the results
  cp_async_wait<0>();
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
            const int c = (i * G + t) * VEC - lead + j;
            if (ANY && (c < 0 || c >= N)) continue;
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
        pg[NP + c] = cols[1][c];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * VEC - lead;
      if (c < N) {
        if (gridDim.x == 1) {
#pragma unroll
          for (int j = 0; j < VEC; ++j)
            if (!ANY || (c + j >= 0 && c + j < N)) {
              if (dgamma) dgamma[c + j] = from_f<WT>(dg[i][j]);
              if (dbeta) dbeta[c + j] = from_f<WT>(db[i][j]);
            }
        } else {  // column c at c + lead: whole vectors, NP being a multiple of VEC
          const int at = c + lead;
#pragma unroll
          for (int j = 0; j < VEC; j += 4) {
            *reinterpret_cast<float4*>(pg + at + j) =
                make_float4(dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]);
            *reinterpret_cast<float4*>(pg + NP + at + j) =
                make_float4(db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]);
          }
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
  const int64_t NP = pad_cols(N);
  float* pg = part + (int64_t)blockIdx.x * 2 * NP;
  for (int64_t c = threadIdx.x; c < N; c += 256) {
    float dg = 0.f, db = 0.f;
    for (int64_t row = blockIdx.x; row < M; row += gridDim.x) {
      const float d = to_f(dy[row * lddy + c]);
      dg += d * ((to_f(x[row * ldx + c]) - mean[row]) * rstd[row]);
      db += d;
    }
    pg[c] = dg;
    pg[NP + c] = db;
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

// dgamma (columns [0, N)) and dbeta (columns [N, 2 N)) = sum of the blocks' partials; block b's
// column c lies at c + (place + b * pitch) % 16 / size. Each of a block's 32 warps sums every 32nd
// partial of 32 columns; the warps' sums are added in order.
template <typename WT>
__global__ void __launch_bounds__(1024) ln_colsum_kernel(const float* __restrict__ part,
                                                         int nparts, int64_t N,
                                                         WT* __restrict__ dgamma,
                                                         WT* __restrict__ dbeta, uint32_t place,
                                                         uint32_t pitch, int size) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane, NP = pad_cols(N);
  float s = 0.f;
  if (c < 2 * N) {
    const float* at = part + (c < N ? c : c - N + NP);
#pragma unroll 5
    for (int b = w; b < nparts; b += 32)
      s += at[(int64_t)b * 2 * NP + ((place + (uint32_t)b * pitch) & 15u) / size];
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

// Every row of one tensor lies in its 16-byte blocks as the same row of the other.
bool same_place(const void* a, int64_t lda, const void* b, int64_t ldb) {
  return ((reinterpret_cast<uintptr_t>(a) ^ reinterpret_cast<uintptr_t>(b)) & 15) == 0 &&
         (lda - ldb) % 16 == 0;
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
  bool wvec;   // gamma and beta lie on 16-byte boundaries
  bool shifted;  // partials of block b lie like row b in its 16-byte blocks
  bool mixed;  // the tensors' rows lie differently in their 16-byte blocks
  cudaStream_t s;
};

// Columns that a row's threads have to hold: with ANY up to V - 1 more, before the first one.
// Tensors whose rows lie differently cannot share a thread's blocks and go the way of the longest
// rows.
template <bool ANY>
int64_t columns(const LnArgs& a, int V) {
  return a.mixed ? INT64_MAX : ANY ? a.N + V - 1 : a.N;
}

template <typename XT, typename WT, bool ANY, int VEC, int G, int PER, int RP = 1>
cudaError_t fwd_launch(const LnArgs& a) {
  constexpr int B = G < 128 ? 128 : G, rows = B / G * RP;
  const int64_t blocks = (a.M + rows - 1) / rows;
  return launch_pdl(ln_fwd_kernel<XT, WT, VEC, G, PER, RP, ANY>, (unsigned)blocks, B, 0, a.s, 1,
                    static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma),
                    static_cast<const WT*>(a.beta), static_cast<XT*>(a.y), a.ldy, a.mean, a.rstd,
                    a.M, (int)a.N, a.eps, (int)a.wvec);
}

// As many blocks as fit at once; their groups' number a multiple of kCycle.
template <typename XT, typename WT, int VEC, int G, int PER>
cudaError_t fwd_walk(const LnArgs& a) {
  constexpr int B = block_of(G), GROUPS = B / G, S = 4, smem = S * PER * B * 16;
  auto kern = ln_fwd_walk_kernel<XT, WT, VEC, G, PER, S>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  static DeviceCache cache;
  const int per_sm = std::max(1, cache.get(current_device(), [&] {
    return blocks_per_sm(reinterpret_cast<const void*>(kern), B, smem);
  }));
  int64_t blocks = std::min<int64_t>((a.M + GROUPS - 1) / GROUPS,
                                     (int64_t)std::max(device_sms(), kCycle) * per_sm);
  if (blocks * GROUPS < a.M) blocks = blocks * GROUPS / kCycle * kCycle / GROUPS;
  return launch_pdl(kern, (unsigned)blocks, B, smem, a.s, 1, static_cast<const XT*>(a.x), a.ldx,
                    static_cast<const WT*>(a.gamma), static_cast<const WT*>(a.beta),
                    static_cast<XT*>(a.y), a.ldy, a.mean, a.rstd, a.M, (int)a.N, a.eps,
                    (int)a.wvec);
}

template <typename XT, typename WT, bool ANY>
cudaError_t fwd_typed(const LnArgs& a) {
  constexpr int V = 16 / sizeof(XT);
  // Weights wider than the rows cost more L1 reads than the rows: two rows share them (16384 x
  // 2880 bf16 rows, fp32 weights: 35.4 us against 42.7). With equal types the registers of a
  // second row cost more than it saves (8192 x 4096 bf16: 29.8 us against 23.2).
  constexpr int RP = sizeof(WT) > sizeof(XT) ? 2 : 1;
  const int64_t N = columns<ANY>(a, V);
  // Up to 32 elements a thread: as few warps a row as hold it, for many rows in flight; with too
  // few rows to fill the GPU that way, as many threads as the row feeds, which is there sooner (300
  // x 4096 bf16: 2.4 us against 2.8; 1200 x 2048: 3.5 against 2.7).
  const bool many = a.M >= (int64_t)std::max(device_sms(), 1) * 2;
  constexpr int P = 32 / V;  // vectors of 32 elements
  if constexpr (ANY) {
    // Many rows: weights moved to the rows' columns once a group. Longer rows, whose groups hold
    // few of them at a time, move them for every row (8192 x 4095 bf16: 55 us against 64), as do
    // few rows.
    if (many) {
      if (N <= 32 * V) return fwd_walk<XT, WT, V, 32, 1>(a);
      if constexpr (V == 4)
        if (N <= 32 * 8) return fwd_walk<XT, WT, V, 32, 2>(a);
      if (N <= 32 * 16) return fwd_walk<XT, WT, V, 32, 16 / V>(a);
      if (N <= 128 * 8) return fwd_walk<XT, WT, V, 128, 8 / V>(a);
      if (N <= 128 * 16) return fwd_walk<XT, WT, V, 128, 16 / V>(a);
      if (N <= 128 * 24) return fwd_walk<XT, WT, V, 128, 24 / V>(a);
      if (N <= 128 * (32 + V)) return fwd_launch<XT, WT, ANY, V, 128, P + 1>(a);
      if (N <= 256 * (32 + V)) return fwd_launch<XT, WT, ANY, V, 256, P + 1>(a);
    }
    if (N <= 32 * V) return fwd_launch<XT, WT, ANY, V, 32, 1>(a);
  } else {
    if (N <= 32 * V) return fwd_launch<XT, WT, ANY, V, 32, 1>(a);
    if (many) {
      if (N <= 32 * 2 * V) return fwd_launch<XT, WT, ANY, V, 32, 2>(a);
      if (N <= 32 * 32) return fwd_launch<XT, WT, ANY, V, 32, P>(a);
      if (N <= 128 * 16) return fwd_launch<XT, WT, ANY, V, 128, P / 2, RP>(a);
      if (N <= 128 * 24) return fwd_launch<XT, WT, ANY, V, 128, P / 4 * 3, RP>(a);
      if (N <= 128 * 32) return fwd_launch<XT, WT, ANY, V, 128, P, RP>(a);
      if (N <= 256 * 32) return fwd_launch<XT, WT, ANY, V, 256, P, RP>(a);
      if (N <= 512 * 32) return fwd_launch<XT, WT, ANY, V, 512, P, RP>(a);
    }
  }
  if (N <= 256 * V) return fwd_launch<XT, WT, ANY, V, 256, 1>(a);
  if (N <= 512 * V) return fwd_launch<XT, WT, ANY, V, 512, 1>(a);
  if (N <= 1024 * V) return fwd_launch<XT, WT, ANY, V, 1024, 1>(a);
  if (N <= 1024 * 16) return fwd_launch<XT, WT, ANY, V, 1024, 16 / V>(a);
  if (N <= 1024 * 32) return fwd_launch<XT, WT, ANY, V, 1024, P>(a);
  const int grid = (int)std::min<int64_t>(a.M, (int64_t)std::max(device_sms(), 1) * 2);
  return launch_pdl(ln_fwd_long_kernel<XT, WT>, grid, 1024, 0, a.s, 1,
                    static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma),
                    static_cast<const WT*>(a.beta), static_cast<XT*>(a.y), a.ldy, a.mean, a.rstd,
                    a.M, a.N, a.eps);
}

template <typename XT, typename WT, bool ANY, int VEC, int G, int PER, int S>
cudaError_t bwd_launch(LnArgs& a) {
  constexpr int B = block_of(G), GROUPS = B / G;
  constexpr int smem = ring_bytes<B, PER, S>();
  auto kern = ln_bwd_kernel<XT, WT, VEC, G, PER, S, ANY>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  // as many blocks as fit at once (at least two where registers allow), each a row of partials
  static DeviceCache cache;
  const int per_sm = std::max(1, cache.get(current_device(), [&] {
    return blocks_per_sm(reinterpret_cast<const void*>(kern), B, smem);
  }));
  const int64_t fit = (int64_t)std::max(device_sms(), 1) * per_sm;
  a.nparts = (int)std::max<int64_t>(
      1, std::min<int64_t>((a.M + GROUPS - 1) / GROUPS, std::min<int64_t>(fit, max_parts(a.N))));
  if (ANY && a.nparts * GROUPS < a.M) a.nparts = a.nparts * GROUPS / kCycle * kCycle / GROUPS;
  a.done = a.nparts == 1;
  a.shifted = ANY && GROUPS == 1;
  return launch_pdl(kern, a.nparts, B, smem, a.s, 1, static_cast<const XT*>(a.dy), a.lddy,
                    static_cast<const XT*>(a.x), a.ldx, static_cast<const WT*>(a.gamma), a.mean,
                    a.rstd, static_cast<XT*>(a.dx), a.lddx, a.part, static_cast<WT*>(a.dgamma),
                    static_cast<WT*>(a.dbeta), a.M, (int)a.N, (int)a.wvec);
}

template <typename XT, typename WT, bool ANY>
cudaError_t bwd_typed(LnArgs& a) {
  constexpr int V = 16 / sizeof(XT);
  const int64_t N = a.N, C = columns<ANY>(a, V);
  if (C <= 32 * V) return bwd_launch<XT, WT, ANY, V, 32, 1, 4>(a);
  if (C <= 32 * 2 * V) return bwd_launch<XT, WT, ANY, V, 32, 2, 3>(a);
  if constexpr (V == 4)
    if (C <= 32 * 16) return bwd_launch<XT, WT, ANY, V, 32, 4, 3>(a);
  if (C <= 128 * 8) return bwd_launch<XT, WT, ANY, V, 128, 8 / V, 4>(a);
  if constexpr (V == 8)
    if (C <= 256 * V) return bwd_launch<XT, WT, ANY, V, 256, 1, 4>(a);
  if (C <= 256 * 2 * V) return bwd_launch<XT, WT, ANY, V, 256, 2, 4>(a);
  if constexpr (sizeof(XT) == 4) {
    if (C <= 256 * 4 * V) return bwd_launch<XT, WT, ANY, V, 256, 4, 3>(a);
  } else {
    if (C <= 512 * 2 * V) return bwd_launch<XT, WT, ANY, V, 512, 2, 3>(a);
  }
  if (C <= 512 * 4 * V) return bwd_launch<XT, WT, ANY, V, 512, 4, 3>(a);
  if constexpr (sizeof(XT) == 4)
    if (C <= 512 * 8 * V) return bwd_launch<XT, WT, ANY, V, 512, 8, 1>(a);
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

// Calls fn with a value of the rows' type, one of the weights', and ANY.
template <class F>
cudaError_t typed(int32_t xd, int32_t wd, bool any, F&& fn) {
  auto with = [&](auto xt, auto wt) {
    return any ? fn(xt, wt, std::true_type()) : fn(xt, wt, std::false_type());
  };
  if (xd == MOE_DT_FP32) return with(float(), float());
  if (wd == MOE_DT_FP32) return with(__nv_bfloat16(), float());
  return with(__nv_bfloat16(), __nv_bfloat16());
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
  a.wvec = aligned_to(gamma, 16) && aligned_to(beta, 16);
  const bool any = !(a.wvec && aligned_to(x, 16) && aligned_to(y, 16) && N * xb % 16 == 0 &&
                     ldx * xb % 16 == 0 && ldy * xb % 16 == 0);
  a.mixed = any && !same_place(x, ldx * xb, y, ldy * xb);
  const cudaError_t e = typed(x_dtype, w_dtype, any, [&](auto xt, auto wt, auto w) {
    return fwd_typed<decltype(xt), decltype(wt), w.value>(a);
  });
  count_launch(a.s, MOE_K_LAYERNORM_FWD);
  if (e != cudaSuccess) return cuda_fail(e, "layernorm forward launch");
  return MOE_OK;
}

size_t moe_layernorm_workspace(int64_t M, int64_t N) {
  if (M < 0 || N < 1 || M > INT32_MAX || N > INT32_MAX) {
    fail(MOE_ERR_INVALID_ARG, "M must be in [0, 2^31) and N in [1, 2^31)");
    return 0;
  }
  return (size_t)std::max<int64_t>(1, std::min<int64_t>(M, max_parts(N))) * 2 * pad_cols(N) *
         sizeof(float);
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
    a.wvec = aligned_to(gamma, 16);
    const bool any = !(a.wvec && aligned_to(x, 16) && aligned_to(dy, 16) && aligned_to(dx, 16) &&
                       N * xb % 16 == 0 && ldx * xb % 16 == 0 && lddy * xb % 16 == 0 &&
                       lddx * xb % 16 == 0);
    a.mixed = any && !(same_place(x, ldx * xb, dy, lddy * xb) &&
                       same_place(x, ldx * xb, dx, lddx * xb));
    e = typed(x_dtype, w_dtype, any, [&](auto xt, auto wt, auto w) {
      return bwd_typed<decltype(xt), decltype(wt), w.value>(a);
    });
    count_launch(a.s, MOE_K_LAYERNORM_BWD);
    if (e != cudaSuccess) return cuda_fail(e, "layernorm backward launch");
  }  // no rows: no partials, the sums are zero
  if (weights && !a.done) {
    const unsigned grid = (unsigned)((2 * N + 31) / 32);
    const uint32_t place = a.shifted ? (uint32_t)(reinterpret_cast<uintptr_t>(x) & 15) : 0u;
    const uint32_t pitch = a.shifted ? (uint32_t)(ldx * xb) : 0u;
    if (w_dtype == MOE_DT_FP32)
      e = launch_pdl(ln_colsum_kernel<float>, grid, 1024, 0, a.s, 1, (const float*)a.part,
                     a.nparts, N, static_cast<float*>(dgamma), static_cast<float*>(dbeta),
                     place, pitch, xb);
    else
      e = launch_pdl(ln_colsum_kernel<__nv_bfloat16>, grid, 1024, 0, a.s, 1,
                     (const float*)a.part, a.nparts, N, static_cast<__nv_bfloat16*>(dgamma),
                     static_cast<__nv_bfloat16*>(dbeta), place, pitch, xb);
    count_launch(a.s, MOE_K_LAYERNORM_REDUCE);
    if (e != cudaSuccess) return cuda_fail(e, "layernorm reduction launch");
  }
  return MOE_OK;
}

}  // extern "C"
