// Load-balance loss of a top-k router, its per-expert counts, and the gradient of the router's
// logits (moe_router_loss_fwd / moe_router_loss_bwd in include/moegmm.h).
//
//   p = softmax(logits) over E;  P_e = mean over valid tokens of p_e;  f_e = E c_e / (k n)
//   loss = coef sum_e f_e P_e
//   d_logits = mask g coef/n p (f - <p, f>)  +  scatter_j w_j (d_j - <w, d>)
//
// Both passes stream the fp32 logits once. A token's row is spread over L lanes of a warp (L the
// power of two that gives each lane one VEC-wide load where it can, so 32/L tokens share a warp),
// and nothing but the row's own E values is kept in registers. Long ones are bound by the latency of
// a row's loads (one row in flight a warp) and by the instructions of a softmax an element (issue
// slots 61 and 75% full), so a row's reductions are straight code; short ones by their launches. Loss
// and gradient with inputs from HBM: 65536 x 256, top 8: 24.0 us (2.9 TB/s; 18.8 us from L2) and
// 26.6 us (5.3 TB/s); 8192 x 8, top 2: 5.7 and 2.1 us; 512 x 4, top 2: 3.8 and 2.5 us.
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;       // gradient
constexpr int kWarps = kThreads / 32;
// Blocks an SM holds, and gets: as many as the registers of eight values a lane allow; more would
// start with the SMs unevenly loaded (65536 x 256: 26.6 us with 5 an SM, 28.3 with 8, 30.7 with 40).
constexpr int kGradBlocks = 5;
constexpr int kLossThreads = 1024;  // loss: one block an SM, so that few partials are left
constexpr int kLossWarps = kLossThreads / 32;
constexpr int kMaxBlocks = 256;     // partial rows the workspace holds
constexpr int kFinishCtas = 8;      // cluster that adds them up, 32 experts a CTA

// One block's share: sum of p over its valid tokens and the pairs routed to the expert. Entry E
// holds the number of valid tokens in c.
struct Partial {
  float p;
  int c;
};

// Row of a token over the lanes of its group: value i*VEC + j of lane `sub` is expert
// (i*L + sub)*VEC + j. NaN and entries past E read as -inf (weight 0 unless the whole row is).
template <int VEC, int V>
MOE_DEVICE void load_row(const float* row, int E, int L, int sub, float (&v)[V * VEC]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = (i * L + sub) * VEC;
    if constexpr (VEC == 4) {
      float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (e < E) q = __ldg(reinterpret_cast<const float4*>(row + e));  // E % 4 == 0
      v[4 * i] = q.x;
      v[4 * i + 1] = q.y;
      v[4 * i + 2] = q.z;
      v[4 * i + 3] = q.w;
    } else {
      v[i] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < V * VEC; ++i) v[i] = fmaxf(v[i], -INFINITY);  // a NaN loses to -inf
}

// Maximum over a group of L lanes; a whole warp's is one instruction (65536 x 256: loss 24.0 us
// against 24.4 with shuffles, gradient 26.6 against 28.0). x is not a NaN.
MOE_DEVICE float group_max(float x, int L) {
  if (L == 32) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
  }
#pragma unroll
  for (int o = L >> 1; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, o));
  return x;
}
MOE_DEVICE float group_sum(float x, int L) {
#pragma unroll
  for (int o = L >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// v <- exp(v - max) over the group; returns the reciprocal of their sum (1 to E). Under an
// infinite maximum the values equal to it weigh 1 and the others 0. expf, as the layer's own
// routing: a power of two with the exponent scaled by a rounded log2(e) would be off by a relative
// |v - max| 2^-24 of a probability.
template <int VEC, int V>
MOE_DEVICE float softmax_row(float (&v)[V * VEC], int E, int L, int sub) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < V * VEC; ++i) m = fmaxf(m, v[i]);
  m = group_max(m, L);
  float s = 0.f;
  if (fabsf(m) < INFINITY) {
#pragma unroll
    for (int i = 0; i < V * VEC; ++i) {
      v[i] = expf(v[i] - m);
      s += v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float& x = v[i * VEC + j];
        x = (i * L + sub) * VEC + j < E && x == m ? 1.0f : 0.f;
        s += x;
      }
  }
  __syncwarp();
  return 1.0f / group_sum(s, L);
}

struct Results {
  float* loss;
  int32_t* counts;
  float* mean_prob;
  int32_t* n_valid;
  double scale;  // coef E / k
};
// Writes an expert's count and mean probability; returns its term of the loss but for scale / n, as
// a pair: the terms are added with more bits than one of them has.
MOE_DEVICE float2 finish_expert(int e, float p, int c, int n, const Results& out) {
  const float mp = n > 0 ? p / (float)n : 0.f;
  out.mean_prob[e] = mp;
  out.counts[e] = c;
  const float x = mp * (float)c;
  return make_float2(x, __fmaf_rn(mp, (float)c, -x));
}
MOE_DEVICE void add_pair(float2& x, float2 y) {
  add_to(x.x, x.y, y.x);
  x.y += y.y;
}
MOE_DEVICE float2 warp_sum(float2 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    add_pair(x, make_float2(__shfl_xor_sync(0xFFFFFFFFu, x.x, o),
                            __shfl_xor_sync(0xFFFFFFFFu, x.y, o)));
  return x;
}
// The loss from the sum of its terms, rounded once. 1/n is fp32's with a step of Newton's method
// in fp64, 46 bits; an fp64 division takes a microsecond of a kernel this short (4096 x 256: 8.6 us
// against 7.3).
MOE_DEVICE float scaled(float2 sum, int n, const Results& out) {
  if (n == 0) return 0.f;
  const double r = 1.0f / (float)n;
  return (float)(((double)sum.x + sum.y) * (out.scale * (r + r * (1.0 - n * r))));
}

// FULL: a token has the whole warp, known when compiling, so that the reductions are straight code.
template <int VEC, int V, bool FULL>
__global__ void __launch_bounds__(kLossThreads) router_loss_kernel(
    const float* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const uint8_t* __restrict__ mask, int T, int E, int k, int lanes, Partial* __restrict__ part,
    const Results out) {
  const int L = FULL ? 32 : lanes;
  MOE_GRIDDEP_ENTRY();
  __shared__ int hist[257];
  __shared__ float psum[kLossWarps][256];
  for (int i = threadIdx.x; i <= E; i += kLossThreads) hist[i] = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (L - 1), grp = lane / L, G = 32 / L;
  const int64_t stride = (int64_t)gridDim.x * kLossWarps * G;
  float acc[V * VEC];
#pragma unroll
  for (int i = 0; i < V * VEC; ++i) acc[i] = 0.f;
  int valid = 0;
  __syncthreads();
  for (int64_t t0 = ((int64_t)blockIdx.x * kLossWarps + warp) * G; t0 < T; t0 += stride) {
    const int64_t t = t0 + grp;
    const bool live = t < T && (!mask || mask[t]);
    const int32_t* id = ids + t * k;
    int e0 = -1;  // this lane's first id, loaded ahead
    if (live && sub < k) e0 = id[sub];
    float v[V * VEC];
    load_row<VEC, V>(logits + (t < T ? t : t0) * ld, E, L, sub, v);
    const float inv = softmax_row<VEC, V>(v, E, L, sub);
    if (live) {
#pragma unroll
      for (int i = 0; i < V * VEC; ++i) acc[i] += v[i] * inv;
      valid += sub == 0;
      if (e0 >= 0 && e0 < E) atomicAdd(&hist[e0], 1);
      for (int j = sub + L; !FULL && j < k; j += L) {
        const int e = id[j];
        if (e >= 0 && e < E) atomicAdd(&hist[e], 1);
      }
    }
    __syncwarp();
  }
  // the warp's token groups, then the block's warps, in a fixed order
#pragma unroll
  for (int i = 0; i < V * VEC; ++i)
    for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], o);
  if (grp == 0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int e = (i * L + sub) * VEC + j;
        if (e < E) psum[warp][e] = acc[i * VEC + j];
      }
  }
  if (valid) atomicAdd(&hist[E], valid);
  __syncthreads();
  Partial o = {0.f, 0};
  const int e = threadIdx.x;  // E < kLossThreads
  if (e <= E) o.c = hist[e];
  if (e < E) {
    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kLossWarps; ++w) s[w & 3] += psum[w][e];
    o.p = (s[0] + s[1]) + (s[2] + s[3]);
  }
  if (gridDim.x > 1) {
    if (e <= E) part[(int64_t)blockIdx.x * (E + 1) + e] = o;
    return;
  }
  // a single block: the results themselves
  __shared__ float2 terms[8];
  const int n = hist[E];
  if (warp * 32 < E) {  // E <= 256
    const float2 x = warp_sum(e < E ? finish_expert(e, o.p, o.c, n, out) : make_float2(0.f, 0.f));
    if (lane == 0) terms[warp] = x;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 x = make_float2(0.f, 0.f);
    for (int w = 0; w * 32 < E; ++w) add_pair(x, terms[w]);
    *out.loss = scaled(x, n, out);
    *out.n_valid = n;
  }
}

// Sums the blocks' partials in a fixed order and forms the loss: one cluster, CTA c for experts
// 32 c .., its warp w for every eighth partial. The sums are pairs of fp32 numbers (65536 x 256:
// fp64 ones, two a cycle and SM, would take 1.2 us): a block's share that fp32 loses beside a
// larger one counts.
__global__ void __launch_bounds__(256)
    router_loss_finish_kernel(const Partial* __restrict__ part, int nblk, int E,
                              const Results out) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sp[8][32], sl[8][32];
  __shared__ int sc[8][32];
  __shared__ int sn[8];
  __shared__ float2 term;
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const uint32_t rank = cluster_ctarank();
  const int e = (int)rank * 32 + lane;
  float p = 0.f, lo = 0.f;
  int c = 0, n = 0;
  if (e < E) {
#pragma unroll 4
    for (int b = w; b < nblk; b += 8) {
      const Partial q = part[(int64_t)b * (E + 1) + e];
      add_to(p, lo, q.p);
      c += q.c;
    }
  }
  for (int b = threadIdx.x; b < nblk; b += 256) n += part[(int64_t)b * (E + 1) + E].c;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xFFFFFFFFu, n, o);
  sp[w][lane] = p;
  sl[w][lane] = lo;
  sc[w][lane] = c;
  if (lane == 0) sn[w] = n;
  __syncthreads();
  n = 0;
  for (int i = 0; i < 8; ++i) n += sn[i];
  if (w == 0) {
    float2 x = make_float2(0.f, 0.f);
    if (e < E) {
      p = lo = 0.f;
      c = 0;
      for (int i = 0; i < 8; ++i) {
        add_to(p, lo, sp[i][lane]);
        lo += sl[i][lane];
        c += sc[i][lane];
      }
      x = finish_expert(e, p + lo, c, n, out);
    }
    x = warp_sum(x);
    if (lane == 0) term = x;
  }
  __syncthreads();
  cluster_sync_all();
  if (rank == 0 && threadIdx.x == 0) {
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (uint32_t r = 0; r < kFinishCtas; ++r) {
      float2 v;
      asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                   : "=f"(v.x), "=f"(v.y) : "r"(mapa_shared(smem_u32(&term), r)) : "memory");
      add_pair(s, v);
    }
    *out.loss = scaled(s, n, out);
    *out.n_valid = n;
  }
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while its term may be read
}

template <int VEC, int V, bool FULL>
__global__ void __launch_bounds__(kThreads, kGradBlocks) router_grad_kernel(
    const float* __restrict__ logits, int64_t ld, const int32_t* __restrict__ ids,
    const float* __restrict__ w, const float* __restrict__ dw, const uint8_t* __restrict__ mask,
    int T, int E, int k, int lanes, float coef, const float* __restrict__ d_loss,
    const int32_t* __restrict__ counts, const int32_t* __restrict__ n_valid,
    float* __restrict__ d, int64_t ldd) {
  MOE_GRIDDEP_ENTRY();
  const int L = FULL ? 32 : lanes;
  // the chosen probabilities' part of a warp's rows, written by slot and read back by expert
  __shared__ __align__(16) float chosen[kWarps][32 * 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane & (L - 1), grp = lane / L, G = 32 / L;
  const int64_t stride = (int64_t)gridDim.x * kWarps * G;
  const int n = *n_valid;
  const float g = n > 0 ? (d_loss ? *d_loss : 1.0f) * coef / (float)n : 0.f;
  const float fs = n > 0 ? (float)E / ((float)k * (float)n) : 0.f;
  for (int i = lane; i < 32 * 8; i += 32) chosen[warp][i] = 0.f;
  float* row_c = &chosen[warp][grp * L * V * VEC];  // G * L * V * VEC <= 256
  float fe[V * VEC];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int e = (i * L + sub) * VEC + j;
      fe[i * VEC + j] = e < E ? fs * (float)counts[e] : 0.f;
    }
  __syncwarp();
  for (int64_t t0 = ((int64_t)blockIdx.x * kWarps + warp) * G; t0 < T; t0 += stride) {
    const int64_t t = t0 + grp;
    const bool in = t < T;
    const int64_t at = t * k + sub;
    int e0 = -1;  // this lane's first slot, loaded ahead
    float w0 = 0.f, d0 = 0.f;
    if (w && in && sub < k) {
      e0 = ids[at];
      w0 = w[at];
      d0 = dw[at];
    }
    float v[V * VEC];
    load_row<VEC, V>(logits + (in ? t : t0) * ld, E, L, sub, v);
    const float inv = softmax_row<VEC, V>(v, E, L, sub);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < V * VEC; ++i) s += v[i] * fe[i];
    s = group_sum(s, L) * inv;
    if (w) {
      const bool ok0 = e0 >= 0 && e0 < E;
      float dot = ok0 ? w0 * d0 : 0.f;
      if (!FULL && in)
        for (int j = L; sub + j < k; j += L) {
          const int e = ids[at + j];
          if (e >= 0 && e < E) dot += w[at + j] * dw[at + j];
        }
      dot = group_sum(dot, L);
      // each slot to its own expert; slots that share one, which a mark left there by each shows,
      // are added in their order
      if (ok0) row_c[e0] = (float)lane;
      __syncwarp();
      const bool shared = (ok0 && row_c[e0] != (float)lane) || (!FULL && k > L);
      if (!__any_sync(0xFFFFFFFFu, shared)) {
        if (ok0) row_c[e0] = w0 * (d0 - dot);
      } else {
        if (ok0) row_c[e0] = 0.f;
        __syncwarp();
        for (int j = 0; j < k; ++j) {
          if (in && sub == j % L) {
            const int e = ids[t * k + j];
            if (e >= 0 && e < E) row_c[e] += w[t * k + j] * (dw[t * k + j] - dot);
          }
          __syncwarp();
        }
      }
      __syncwarp();
    }
    const float c = in && (!mask || mask[t]) ? g : 0.f;
    const float ci = c * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = (i * L + sub) * VEC;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int q = i * VEC + j;
        o[j] = ci * v[q] * (fe[q] - s);  // a masked row's factors are finite, its ci is 0
      }
      if (e < E) {
        if constexpr (VEC == 4) {
          if (w) {
            float4& r = *reinterpret_cast<float4*>(row_c + e);
            o[0] += r.x;
            o[1] += r.y;
            o[2] += r.z;
            o[3] += r.w;
            r = make_float4(0.f, 0.f, 0.f, 0.f);
          }
          if (in) *reinterpret_cast<float4*>(d + t * ldd + e) = make_float4(o[0], o[1], o[2], o[3]);
        } else {
          if (w) {
            o[0] += row_c[e];
            row_c[e] = 0.f;
          }
          if (in) d[t * ldd + e] = o[0];
        }
      }
    }
    __syncwarp();
  }
}

// Lanes a token's row is spread over and loads per lane.
struct RowMap {
  int vec, L, V;
};
RowMap row_map(int E, bool vec4) {
  RowMap m;
  m.vec = vec4 ? 4 : 1;
  const int words = (E + m.vec - 1) / m.vec;
  m.L = 1;
  while (m.L < words && m.L < 32) m.L <<= 1;
  const int v = (words + m.L - 1) / m.L;
  m.V = v <= 1 ? 1 : v <= 2 ? 2 : v <= 4 ? 4 : 8;
  return m;
}

// Calls fn with the kernel's template arguments as integral constants.
template <int N>
using I = std::integral_constant<int, N>;
template <class F>
void with_map(const RowMap& m, F&& fn) {
  if (m.vec == 4) {
    if (m.L < 32) fn(I<4>(), I<1>(), std::false_type());
    else if (m.V == 1) fn(I<4>(), I<1>(), std::true_type());
    else fn(I<4>(), I<2>(), std::true_type());
  } else if (m.L < 32) {
    fn(I<1>(), I<1>(), std::false_type());
  } else if (m.V == 1) {
    fn(I<1>(), I<1>(), std::true_type());
  } else if (m.V == 2) {
    fn(I<1>(), I<2>(), std::true_type());
  } else if (m.V == 4) {
    fn(I<1>(), I<4>(), std::true_type());
  } else {
    fn(I<1>(), I<8>(), std::true_type());
  }
}

int router_blocks(int64_t T, const RowMap& m, int warps, int most) {
  const int64_t per_block = (int64_t)warps * (32 / m.L);
  return (int)std::max<int64_t>(1, std::min<int64_t>((T + per_block - 1) / per_block, most));
}

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

moe_status_t check_sizes(int32_t T, int32_t E, int32_t k, int64_t ld) {
  if (E < 1 || E > 256) return fail(MOE_ERR_INVALID_ARG, "E=%d outside [1,256]", E);
  if (k < 1 || k > 8 || k > E)
    return fail(MOE_ERR_INVALID_ARG, "k=%d must be in [1, min(E,8)]", k);
  if (T < 0) return fail(MOE_ERR_INVALID_ARG, "T=%d is negative", T);
  if (ld < E) return fail(MOE_ERR_INVALID_ARG, "ld_logits must be >= E");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_router_loss_workspace(int32_t E) {
  if (E < 1 || E > 256) {
    fail(MOE_ERR_INVALID_ARG, "E=%d outside [1,256]", E);
    return 0;
  }
  return (size_t)kMaxBlocks * (E + 1) * sizeof(Partial);
}

moe_status_t moe_router_loss_fwd(const float* logits, int64_t ld_logits, const int32_t* topk_ids,
                                 const uint8_t* token_mask, int32_t T, int32_t E, int32_t k,
                                 float coef, float* loss, int32_t* counts, float* mean_prob,
                                 int32_t* n_valid, void* ws, size_t ws_bytes,
                                 moe_stream_t stream) {
  moe_status_t st = check_sizes(T, E, k, ld_logits);
  if (st != MOE_OK) return st;
  if ((T > 0 && (!logits || !topk_ids)) || !loss || !counts || !mean_prob || !n_valid || !ws)
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!a4(logits) || !a4(topk_ids) || !a4(loss) || !a4(counts) || !a4(mean_prob) || !a4(n_valid))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be 4-byte aligned");
  if (!a16(ws)) return fail(MOE_ERR_INVALID_ARG, "ws must be 16-byte aligned");
  if (ws_bytes < moe_router_loss_workspace(E))
    return fail(MOE_ERR_WORKSPACE, "ws_bytes=%zu < required %zu", ws_bytes,
                moe_router_loss_workspace(E));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RowMap m = row_map(E, E % 4 == 0 && ld_logits % 4 == 0 && a16(logits));
  // up to four turns of one block: about as soon done as two launches (2048 x 8, four turns: 6.2 us
  // against 5.4; 4096 x 8, eight: 9.4 against 5.8), and 2 us less on the host
  int nblk = router_blocks(T, m, kLossWarps, std::min(std::max(device_sms(), 1), kMaxBlocks));
  if (nblk <= 4) nblk = 1;
  const Results out = {loss, counts, mean_prob, n_valid, (double)coef * E / k};
  Partial* part = static_cast<Partial*>(ws);
  cudaError_t e = cudaSuccess;
  with_map(m, [&](auto vec, auto v, auto full) {
    e = launch_pdl(router_loss_kernel<vec.value, v.value, full.value>, nblk, kLossThreads, 0, s, 1,
                   logits, ld_logits, topk_ids, token_mask, T, E, k, m.L, part, out);
  });
  count_launch(s, MOE_K_ROUTER_LOSS);
  if (e != cudaSuccess) return cuda_fail(e, "router loss launch");
  if (nblk == 1) return MOE_OK;
  e = launch_pdl(router_loss_finish_kernel, kFinishCtas, 256, 0, s, kFinishCtas,
                 (const Partial*)part, nblk, E, out);
  count_launch(s, MOE_K_ROUTER_LOSS);
  if (e != cudaSuccess) return cuda_fail(e, "router loss finish launch");
  return MOE_OK;
}

moe_status_t moe_router_loss_bwd(const float* logits, int64_t ld_logits, const int32_t* topk_ids,
                                 const float* topk_probs, const float* d_probs,
                                 const uint8_t* token_mask, int32_t T, int32_t E, int32_t k,
                                 float coef, const float* d_loss, const int32_t* counts,
                                 const int32_t* n_valid, float* d_logits, int64_t ld_d,
                                 moe_stream_t stream) {
  moe_status_t st = check_sizes(T, E, k, ld_logits);
  if (st != MOE_OK) return st;
  if (ld_d < E) return fail(MOE_ERR_INVALID_ARG, "ld_d must be >= E");
  if ((topk_probs != nullptr) != (d_probs != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "topk_probs and d_probs go together");
  if (!counts || !n_valid || (T > 0 && (!logits || !topk_ids || !d_logits)))
    return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  if (!a4(logits) || !a4(topk_ids) || !a4(topk_probs) || !a4(d_probs) || !a4(d_loss) ||
      !a4(counts) || !a4(n_valid) || !a4(d_logits))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be 4-byte aligned");
  if (T == 0) return MOE_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const RowMap m = row_map(E, E % 4 == 0 && ld_logits % 4 == 0 && ld_d % 4 == 0 && a16(logits) &&
                                  a16(d_logits));
  const int nblk = router_blocks(T, m, kWarps, std::max(device_sms(), 1) * kGradBlocks);
  cudaError_t e = cudaSuccess;
  with_map(m, [&](auto vec, auto v, auto full) {
    e = launch_pdl(router_grad_kernel<vec.value, v.value, full.value>, nblk, kThreads, 0, s, 1,
                   logits, ld_logits, topk_ids, topk_probs, d_probs, token_mask, T, E, k, m.L,
                   coef, d_loss, counts, n_valid, d_logits, ld_d);
  });
  count_launch(s, MOE_K_ROUTER_GRAD);
  if (e != cudaSuccess) return cuda_fail(e, "router gradient launch");
  return MOE_OK;
}

}  // extern "C"
