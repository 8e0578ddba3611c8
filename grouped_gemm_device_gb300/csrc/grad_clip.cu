// Global gradient norm over a list of tensors, and clipping (moe_grad_clip in
// include/moegmm.h).
//
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c g
//
// Bound by HBM: one read of every gradient for the norm, one read and one write for the product.
// 1.41 G bf16 elements 1250 us (6.7 TB/s over the three passes, the measured copy rate), 20 M 22
// us (17 with its inputs in L2), 60 k fp32 3.9 us in place and not clipped. Two kinds of launch:
// partial sums (one a block), then the product, whose blocks each add up the partial sums in the
// same order, so that no launch, counter or atomic joins them.
// Sums are pairs of fp32 numbers (a running sum and what its roundings lost, by the error-free sum
// of two numbers, Knuth 1969): about 48 bits at the full fp32 rate, where this GPU adds two fp64
// numbers an SM and cycle. Squares that fp32 cannot hold go into an fp64 sum of their own.
// The tensors travel as kernel parameters (up to kCap a launch); their elements are cut into
// chunks that blocks take in turn.
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 4;                          // 16-byte loads a thread and chunk
constexpr int kChunkBytes = kThreads * kVecs * 16;
constexpr int kCap = 96;                          // tensors a launch
constexpr int kMaxBlocks = 1216;                  // partial sums one launch leaves
constexpr int kMaxParts = 32768;                  // partial sums all launches leave together
constexpr float kEps = 1e-6f;

// A tensor is cut at 16-byte boundaries of its address: `src` is rounded down to one, `lead` the
// elements before the first, so that element i sits at src[lead + i].
struct Tensor {
  const void* src;
  void* dst;
  int64_t numel;
  int64_t first_chunk;
  int16_t fp32, lead, dst_vec, unused;
};
struct Batch {
  Tensor t[kCap];
  int n;
  int64_t chunks;
};

MOE_DEVICE int find_tensor(const Batch& b, int64_t chunk) {
  int lo = 0, hi = b.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (b.t[mid].first_chunk <= chunk) lo = mid; else hi = mid;
  }
  return lo;
}

// The 16 bytes of vector `v` (element index v * PER of the rounded-down tensor); elements outside
// [lead, lead + numel) read as 0.
template <int PER>
MOE_DEVICE uint4 load16(const Tensor& t, int64_t v) {
  const int64_t e = v * PER, end = t.lead + t.numel;
  uint32_t u[4] = {0u, 0u, 0u, 0u};
  if (e >= t.lead && e + PER <= end) return reinterpret_cast<const uint4*>(t.src)[v];
  if (e < end) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (e + i < t.lead || e + i >= end) continue;
      if constexpr (PER == 8)
        u[i >> 1] |= (uint32_t)static_cast<const uint16_t*>(t.src)[e + i] << (16 * (i & 1));
      else
        u[i] = static_cast<const uint32_t*>(t.src)[e + i];
    }
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}
template <int PER>
MOE_DEVICE void widen(const uint4& q, float (&x)[PER]) {
  const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (PER == 8) {
      x[2 * i] = bf16_lo(u[i]);
      x[2 * i + 1] = bf16_hi(u[i]);
    } else {
      x[i] = __uint_as_float(u[i]);
    }
  }
}

// hi + lo, and what lies outside fp32's comfortable range.
struct Sum {
  float hi, lo;
  double odd;
};

// Adds the squares of one thread's share of a chunk: at most 32 of them in fp32 where their sum
// is well inside its range; otherwise (an overflow, a NaN, or squares that may have been lost
// below the range) in fp64.
template <int PER>
MOE_DEVICE void add_squares(const Tensor& t, int64_t v0, Sum& sum) {
  uint4 q[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) q[i] = load16<PER>(t, v0 + i * kThreads);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float x[PER], p = 0.f;
    widen<PER>(q[i], x);
#pragma unroll
    for (int j = 0; j < PER; ++j) p += x[j] * x[j];
    s += p;
  }
  if (s > 1e-20f && s < 1e28f) {
    add_to(sum.hi, sum.lo, s);
    return;
  }
  uint32_t any = 0;  // an expert without tokens has zero gradients: nothing to add
#pragma unroll
  for (int i = 0; i < kVecs; ++i) any |= q[i].x | q[i].y | q[i].z | q[i].w;
  if (any == 0) return;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float x[PER];
    widen<PER>(q[i], x);
#pragma unroll 1
    for (int j = 0; j < PER; ++j) sum.odd += (double)x[j] * (double)x[j];
  }
}

// The block's sum, the same in every thread.
MOE_DEVICE Sum block_sum(Sum v) {
  __shared__ float s_hi[kThreads / 32], s_lo[kThreads / 32];
  __shared__ double s_odd[kThreads / 32];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xFFFFFFFFu, v.hi, o);
    const float lo = __shfl_xor_sync(0xFFFFFFFFu, v.lo, o);
    add_to(v.hi, v.lo, hi);
    v.lo += lo;
  }
  if (lane == 0) {
    s_hi[w] = v.hi;
    s_lo[w] = v.lo;
  }
  const bool odd = __syncthreads_or(v.odd != 0.0);  // also a barrier for the sums above
  v.hi = v.lo = 0.f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    add_to(v.hi, v.lo, s_hi[i]);
    v.lo += s_lo[i];
  }
  if (odd) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v.odd += __shfl_xor_sync(0xFFFFFFFFu, v.odd, o);
    if (lane == 0) s_odd[w] = v.odd;
    __syncthreads();
    v.odd = 0.0;
    for (int i = 0; i < kThreads / 32; ++i) v.odd += s_odd[i];
  }
  return v;
}

// One thread's share of the partial sums.
MOE_DEVICE Sum sum_parts(const Sum* part, int nparts) {
  Sum s = {0.f, 0.f, 0.0};
  for (int i = threadIdx.x; i < nparts; i += kThreads) {
    const Sum p = part[i];
    add_to(s.hi, s.lo, p.hi);
    s.lo += p.lo;
    if (p.odd != 0.0) s.odd += p.odd;
  }
  return s;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Batch b,
                                                             Sum* __restrict__ part) {
  MOE_GRIDDEP_ENTRY();
  Sum s = {0.f, 0.f, 0.0};
  for (int64_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const Tensor& t = b.t[find_tensor(b, c)];
    const int64_t v0 = (c - t.first_chunk) * (kThreads * kVecs) + threadIdx.x;
    if (t.fp32) add_squares<4>(t, v0, s);
    else add_squares<8>(t, v0, s);
  }
  s = block_sum(s);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// The factor as a product: `once` alone, and `again` 1, unless it is below fp32's normal numbers.
struct Factor {
  float once, again;
};
template <int PER, bool AGAIN>
MOE_DEVICE void scale_chunk(const Tensor& t, int64_t v0, Factor c) {
  uint4 q[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) q[i] = load16<PER>(t, v0 + i * kThreads);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    const int64_t e = (v0 + i * kThreads) * PER, end = t.lead + t.numel;
    if (e >= end) continue;
    float x[PER];
    widen<PER>(q[i], x);
#pragma unroll
    for (int j = 0; j < PER; ++j) x[j] = AGAIN ? (x[j] * c.once) * c.again : x[j] * c.once;
    // dst counts elements from the tensor's own first one
    if (t.dst_vec && e >= t.lead && e + PER <= end) {
      if constexpr (PER == 8)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(t.dst) + (e - t.lead)) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                       pack_bf16x2(x[6], x[7]));
      else
        *reinterpret_cast<float4*>(static_cast<float*>(t.dst) + (e - t.lead)) =
            make_float4(x[0], x[1], x[2], x[3]);
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (e + j < t.lead || e + j >= end) continue;
        if constexpr (PER == 8)
          static_cast<__nv_bfloat16*>(t.dst)[e + j - t.lead] = __float2bfloat16_rn(x[j]);
        else
          static_cast<float*>(t.dst)[e + j - t.lead] = x[j];
      }
    }
  }
}

// AGAIN: a second factor. A loop of its own: in the usual one its product costs 17.6 us against 17.2
// (20 M bf16).
template <bool AGAIN>
MOE_DEVICE void scale_chunks(const Batch& b, Factor c) {
  // last chunks first: they are what the norm's pass read last, and may still be in L2
  for (int64_t q = b.chunks - 1 - blockIdx.x; q >= 0; q -= gridDim.x) {
    const Tensor& t = b.t[find_tensor(b, q)];
    const int64_t v0 = (q - t.first_chunk) * (kThreads * kVecs) + threadIdx.x;
    if (t.fp32) scale_chunk<4, AGAIN>(t, v0, c);
    else scale_chunk<8, AGAIN>(t, v0, c);
  }
}

// Several launches' partial sums into one (one block).
__global__ void __launch_bounds__(kThreads) grad_total_kernel(const Sum* __restrict__ part,
                                                              int nparts, Sum* __restrict__ total) {
  MOE_GRIDDEP_ENTRY();
  const Sum s = block_sum(sum_parts(part, nparts));
  if (threadIdx.x == 0) *total = s;
}

// c = min(1, max_norm / (norm + eps)) in fp32; a NaN norm gives NaN. A finite norm that fp32 cannot
// hold (four elements of 3e38 have one) divides in fp64, and a subnormal factor is 2^-64 times one
// with all its bits: |x| c 2^64 stays below 2^66.
MOE_DEVICE Factor clip_factor(const Sum& s, float norm, float max_norm) {
  if (norm == INFINITY) {
    const double exact = sqrt(((double)s.hi + (double)s.lo) + s.odd);
    if (exact < INFINITY) {
      const double r = max_norm / exact;
      return r < 0x1p-126 ? Factor{(float)(r * 0x1p64), 0x1p-64f} : Factor{(float)r, 1.0f};
    }
  }
  const float r = max_norm / (norm + kEps);
  return {r >= 1.0f ? 1.0f : r, 1.0f};
}

// in_place: nothing to do when the factor is 1. apply = 0: only the norm.
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ Batch b,
                                                              const Sum* __restrict__ part,
                                                              int nparts, float max_norm,
                                                              int apply, int in_place,
                                                              float* __restrict__ norm_out) {
  MOE_GRIDDEP_ENTRY();
  const Sum s = block_sum(sum_parts(part, nparts));
  const float norm = s.odd != 0.0 ? (float)sqrt(((double)s.hi + (double)s.lo) + s.odd)
                                  : sqrtf(s.hi + s.lo);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  if (!apply) return;
  const Factor c = clip_factor(s, norm, max_norm);
  if (in_place && c.once == 1.0f) return;
  if (c.again == 1.0f) scale_chunks<false>(b, c);
  else scale_chunks<true>(b, c);
}

// Tensors [i, i + kCap) of the list that hold elements; returns the next index.
int fill_batch(Batch& b, int i, int n, const void* const* grads, void* const* outs,
               const int64_t* numel, const int32_t* dtypes) {
  b.n = 0;
  b.chunks = 0;
  for (; i < n && b.n < kCap; ++i) {
    if (numel[i] == 0) continue;
    Tensor& t = b.t[b.n++];
    const int es = dtypes[i] == MOE_DT_FP32 ? 4 : 2;
    const uintptr_t p = reinterpret_cast<uintptr_t>(grads[i]);
    void* dst = outs ? outs[i] : const_cast<void*>(grads[i]);
    t.src = reinterpret_cast<const void*>(p & ~(uintptr_t)15);
    t.dst = dst;
    t.numel = numel[i];
    t.fp32 = es == 4;
    t.lead = (int16_t)((p & 15) / es);
    t.dst_vec = ((reinterpret_cast<uintptr_t>(dst) ^ p) & 15) == 0;
    t.unused = 0;
    t.first_chunk = b.chunks;
    b.chunks += ((t.lead + numel[i]) * es + kChunkBytes - 1) / kChunkBytes;
  }
  return i;
}

// As many blocks as fit at once, or one a chunk. Very long lists get twice as many, which evens
// out the blocks' ends (1.4 G bf16 elements: 1247 us against 1301; at 20 M the second half only
// costs its start, 21.5 us against 18.2).
template <class K>
int clip_blocks(K kernel, int64_t chunks) {
  static DeviceCache cache;
  const int per_sm = std::max(1, cache.get(current_device(), [&] {
    return blocks_per_sm(reinterpret_cast<const void*>(kernel), kThreads, 0);
  }));
  const int64_t fit = (int64_t)std::max(device_sms(), 1) * per_sm;
  const int64_t most = std::min<int64_t>(kMaxBlocks, chunks > 64 * fit ? 2 * fit : fit);
  return (int)std::max<int64_t>(1, std::min(chunks, most));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grad_clip_workspace(void) {
  return (size_t)(kMaxParts + 1) * sizeof(Sum);
}

moe_status_t moe_grad_clip(int32_t n, const void* const* grads, void* const* outs,
                           const int64_t* numel, const int32_t* dtypes, float max_norm,
                           float* norm, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (n < 0 || n > 65536) return fail(MOE_ERR_INVALID_ARG, "n=%d outside [0, 65536]", n);
  if (n > 0 && (!grads || !numel || !dtypes)) return fail(MOE_ERR_INVALID_ARG, "NULL host array");
  if (!(max_norm > 0.f)) return fail(MOE_ERR_INVALID_ARG, "max_norm must be > 0");
  const bool apply = max_norm <= 3.402823466e38f;
  if (!apply && outs)
    return fail(MOE_ERR_INVALID_ARG, "outs must be NULL when max_norm is infinite");
  if (!norm || !ws) return fail(MOE_ERR_INVALID_ARG, "NULL norm or ws");
  if ((reinterpret_cast<uintptr_t>(norm) & 3) || (reinterpret_cast<uintptr_t>(ws) & 15))
    return fail(MOE_ERR_INVALID_ARG, "norm must be 4-byte and ws 16-byte aligned");
  if (ws_bytes < moe_grad_clip_workspace())
    return fail(MOE_ERR_WORKSPACE, "ws_bytes=%zu < required %zu", ws_bytes,
                moe_grad_clip_workspace());
  for (int i = 0; i < n; ++i) {
    if (dtypes[i] != MOE_DT_BF16 && dtypes[i] != MOE_DT_FP32)
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: unknown dtype %d", i, dtypes[i]);
    if (numel[i] < 0) return fail(MOE_ERR_INVALID_ARG, "tensor %d: negative size", i);
    if (numel[i] == 0) continue;
    const uintptr_t es = dtypes[i] == MOE_DT_FP32 ? 4 : 2;
    const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
    const uintptr_t o = outs ? reinterpret_cast<uintptr_t>(outs[i]) : g;
    if (!g || !o) return fail(MOE_ERR_INVALID_ARG, "tensor %d: NULL pointer", i);
    if (g % es || o % es)
      return fail(MOE_ERR_INVALID_ARG, "tensor %d: not aligned to its elements", i);
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Sum* part = static_cast<Sum*>(ws);
  int nparts = 0, held = 0, batches = 0;
  for (int i = 0; i < n; ++i) held += numel[i] != 0;
  // few launches take as many blocks as fit; many share the room for their partial sums
  const int launches = (held + kCap - 1) / kCap;
  const int most = launches > 0 ? std::max(kMaxParts / launches, 1) : 1;
  bool in_place = true;
  for (int i = 0; outs && i < n; ++i) in_place = in_place && (outs[i] == grads[i] || !numel[i]);
  Batch b;
  cudaError_t e;
  for (int i = 0; i < n;) {
    i = fill_batch(b, i, n, grads, outs, numel, dtypes);
    if (b.n == 0) break;
    const int grid = std::min(clip_blocks(grad_norm_kernel, b.chunks), most);
    e = launch_pdl(grad_norm_kernel, grid, kThreads, 0, s, 1, b, part + nparts);
    count_launch(s, MOE_K_GRAD_NORM);
    if (e != cudaSuccess) return cuda_fail(e, "gradient norm launch");
    nparts += grid;
    ++batches;
  }
  if (batches > 1) {
    e = launch_pdl(grad_total_kernel, 1, kThreads, 0, s, 1, (const Sum*)part, nparts,
                       part + kMaxParts);
    count_launch(s, MOE_K_GRAD_NORM);
    if (e != cudaSuccess) return cuda_fail(e, "gradient norm total launch");
    part += kMaxParts;
    nparts = 1;
  }
  // the batches once more; every launch forms the same norm and factor
  int written = 0;
  for (int i = 0; i < n || written == 0;) {
    i = fill_batch(b, i, n, grads, outs, numel, dtypes);
    if (b.n == 0 && written > 0) break;
    const int grid = apply ? clip_blocks(grad_scale_kernel, b.chunks) : 1;
    e = launch_pdl(grad_scale_kernel, grid, kThreads, 0, s, 1, b, (const Sum*)part, nparts,
                       max_norm, apply ? 1 : 0, in_place ? 1 : 0, written == 0 ? norm : nullptr);
    count_launch(s, MOE_K_GRAD_SCALE);
    if (e != cudaSuccess) return cuda_fail(e, "gradient scale launch");
    ++written;
    if (!apply) break;
  }
  return MOE_OK;
}

}  // extern "C"
