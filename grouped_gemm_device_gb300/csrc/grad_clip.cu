// Global gradient norm over a list of tensors, and clipping (moe_grad_clip in
// include/moegmm.h).
//
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c g
//
// Bound by HBM: one read of every gradient for the norm, one read and one write for the product.
// Two kinds of launch: partial sums (one fp64 value a block), then the product, whose blocks each
// add up the partial sums in the same order, so that no launch, counter or atomic joins them.
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
constexpr int kMaxLaunches = (65536 + kCap - 1) / kCap;
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

// The 16 bytes of vector `v` (element index v * PER of the rounded-down tensor) as fp32; elements
// outside [lead, lead + numel) read as 0.
template <int PER>
MOE_DEVICE bool load16(const Tensor& t, int64_t v, float (&x)[PER]) {
  const int64_t e = v * PER, end = t.lead + t.numel;
  if (e >= end) {
#pragma unroll
    for (int i = 0; i < PER; ++i) x[i] = 0.f;
    return false;
  }
  if (e >= t.lead && e + PER <= end) {
    const uint4 q = reinterpret_cast<const uint4*>(t.src)[v];
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
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool in = e + i >= t.lead && e + i < end;
      if constexpr (PER == 8)
        x[i] = in ? __bfloat162float(static_cast<const __nv_bfloat16*>(t.src)[e + i]) : 0.f;
      else
        x[i] = in ? static_cast<const float*>(t.src)[e + i] : 0.f;
    }
  }
  return true;
}

// Sum of squares of one thread's share of a chunk. fp32 where the result is well inside its
// range; otherwise (an overflow, or squares that may have been lost below it) fp64.
template <int PER>
MOE_DEVICE double chunk_squares(const Tensor& t, int64_t v0) {
  float x[kVecs][PER];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) load16<PER>(t, v0 + i * kThreads, x[i]);
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < PER; ++j) q += x[i][j] * x[i][j];
    s += q;
  }
  if (s > 1e-20f && s < 1e30f) return (double)s;
  bool zero = s == 0.f;  // an expert without tokens has zero gradients: nothing to add
#pragma unroll
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int j = 0; j < PER; ++j) zero = zero && x[i][j] == 0.f;
  if (zero) return 0.0;
  double d = 0.0;
#pragma unroll 1
  for (int i = 0; i < kVecs; ++i)
#pragma unroll
    for (int j = 0; j < PER; ++j) d += (double)x[i][j] * (double)x[i][j];
  return d;
}

MOE_DEVICE double block_sum(double v, double* sm) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += sm[w];
  return s;
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ Batch b,
                                                             double* __restrict__ part) {
  MOE_GRIDDEP_ENTRY();
  __shared__ double sm[kThreads / 32];
  double s = 0.0;
  for (int64_t c = blockIdx.x; c < b.chunks; c += gridDim.x) {
    const Tensor& t = b.t[find_tensor(b, c)];
    const int64_t v0 = (c - t.first_chunk) * (kThreads * kVecs) + threadIdx.x;
    s += t.fp32 ? chunk_squares<4>(t, v0) : chunk_squares<8>(t, v0);
  }
  s = block_sum(s, sm);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

template <int PER>
MOE_DEVICE void scale_chunk(const Tensor& t, int64_t v0, float c) {
  float x[kVecs][PER];
  bool in[kVecs];
#pragma unroll
  for (int i = 0; i < kVecs; ++i) in[i] = load16<PER>(t, v0 + i * kThreads, x[i]);
#pragma unroll
  for (int i = 0; i < kVecs; ++i) {
    if (!in[i]) continue;
    const int64_t e = (v0 + i * kThreads) * PER, end = t.lead + t.numel;
#pragma unroll
    for (int j = 0; j < PER; ++j) x[i][j] *= c;
    // dst counts elements from the tensor's own first one
    if (t.dst_vec && e >= t.lead && e + PER <= end) {
      uint4 q;
      if constexpr (PER == 8)
        q = make_uint4(pack_bf16x2(x[i][0], x[i][1]), pack_bf16x2(x[i][2], x[i][3]),
                       pack_bf16x2(x[i][4], x[i][5]), pack_bf16x2(x[i][6], x[i][7]));
      else
        q = make_uint4(__float_as_uint(x[i][0]), __float_as_uint(x[i][1]),
                       __float_as_uint(x[i][2]), __float_as_uint(x[i][3]));
      if constexpr (PER == 8)
        *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(t.dst) + (e - t.lead)) = q;
      else
        *reinterpret_cast<uint4*>(static_cast<float*>(t.dst) + (e - t.lead)) = q;
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        if (e + j < t.lead || e + j >= end) continue;
        if constexpr (PER == 8)
          static_cast<__nv_bfloat16*>(t.dst)[e + j - t.lead] = __float2bfloat16_rn(x[i][j]);
        else
          static_cast<float*>(t.dst)[e + j - t.lead] = x[i][j];
      }
    }
  }
}

// c = min(1, max_norm / (norm + eps)) in fp32; a NaN norm gives NaN.
MOE_DEVICE float clip_factor(float norm, float max_norm) {
  const float r = max_norm / (norm + kEps);
  return r >= 1.0f ? 1.0f : r;
}

// in_place: nothing to do when the factor is 1. apply = 0: only the norm.
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ Batch b,
                                                              const double* __restrict__ part,
                                                              int nparts, float max_norm,
                                                              int apply, int in_place,
                                                              float* __restrict__ norm_out) {
  MOE_GRIDDEP_ENTRY();
  __shared__ double sm[kThreads / 32];
  double s = 0.0;
  for (int i = threadIdx.x; i < nparts; i += kThreads) s += part[i];
  s = block_sum(s, sm);
  const float norm = (float)sqrt(s);
  if (norm_out && blockIdx.x == 0 && threadIdx.x == 0) *norm_out = norm;
  if (!apply) return;
  const float c = clip_factor(norm, max_norm);
  if (in_place && c == 1.0f) return;
  // last chunks first: they are what the norm's pass read last, and may still be in L2
  for (int64_t q = b.chunks - 1 - blockIdx.x; q >= 0; q -= gridDim.x) {
    const Tensor& t = b.t[find_tensor(b, q)];
    const int64_t v0 = (q - t.first_chunk) * (kThreads * kVecs) + threadIdx.x;
    if (t.fp32) scale_chunk<4>(t, v0, c);
    else scale_chunk<8>(t, v0, c);
  }
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

int clip_blocks(int64_t chunks) {
  const int64_t most = std::min<int64_t>(kMaxBlocks, (int64_t)std::max(device_sms(), 1) * 8);
  return (int)std::max<int64_t>(1, std::min(chunks, most));
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grad_clip_workspace(void) {
  return (size_t)kMaxBlocks * kMaxLaunches * sizeof(double);
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
  double* part = static_cast<double*>(ws);
  int nparts = 0;
  bool in_place = true;
  for (int i = 0; outs && i < n; ++i) in_place = in_place && (outs[i] == grads[i] || !numel[i]);
  Batch b;
  cudaError_t e;
  for (int i = 0; i < n;) {
    i = fill_batch(b, i, n, grads, outs, numel, dtypes);
    if (b.n == 0) break;
    const int grid = clip_blocks(b.chunks);
    if (nparts == 0) {
      grad_norm_kernel<<<grid, kThreads, 0, s>>>(b, part);
      e = cudaGetLastError();
    } else {
      e = launch_chained(grad_norm_kernel, grid, kThreads, 0, s, b, part + nparts);
    }
    count_launch(s, MOE_K_GRAD_NORM);
    if (e != cudaSuccess) return cuda_fail(e, "gradient norm launch");
    nparts += grid;
  }
  // the batches once more; every launch forms the same norm and factor
  int written = 0;
  for (int i = 0; i < n || written == 0;) {
    i = fill_batch(b, i, n, grads, outs, numel, dtypes);
    if (b.n == 0 && written > 0) break;
    const int grid = apply ? clip_blocks(b.chunks) : 1;
    e = launch_chained(grad_scale_kernel, grid, kThreads, 0, s, b, (const double*)part, nparts,
                       max_norm, apply ? 1 : 0, in_place ? 1 : 0, written == 0 ? norm : nullptr);
    count_launch(s, MOE_K_GRAD_SCALE);
    if (e != cudaSuccess) return cuda_fail(e, "gradient scale launch");
    ++written;
    if (!apply) break;
  }
  return MOE_OK;
}

}  // extern "C"
