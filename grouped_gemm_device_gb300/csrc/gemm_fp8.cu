// Dense product of E4M3 operands with an fp32 scale for each block of 128 (fp8_block_gemm in
// include/moegmm.h): C = sum over k-blocks of sa * sb * (a_block . b_block^T).
//
// Plain version: a 64 x 64 tile a block, both operands widened to fp32 in shared memory, one
// fp32 accumulator for the current k-block and one for the result.
#include "kernels.cuh"

#include <cuda_fp8.h>

namespace moe {
namespace {

constexpr int kBM = 64, kBN = 64, kBK = 32, kThreads = 256;

struct Fp8Args {
  const uint8_t *a, *b;
  int64_t lda, ldb;
  const float *sa, *sb;
  int64_t ld_sa, ld_sb;
  int b_block;
  void* c;
  int64_t ldc;
  int c_fp32;
  int64_t M, N, K;
};

MOE_DEVICE float e4m3_to_f(uint8_t q) {
  __nv_fp8_e4m3 v;
  v.__x = q;
  return float(v);
}

__global__ void __launch_bounds__(kThreads) fp8_gemm_plain_kernel(const Fp8Args p) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sA[kBK][kBM + 1], sB[kBK][kBN + 1];
  const int64_t m0 = (int64_t)blockIdx.y * kBM, n0 = (int64_t)blockIdx.x * kBN;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {}, part[4][4] = {};
  for (int64_t k0 = 0; k0 < p.K; k0 += kBK) {
    for (int i = threadIdx.x; i < kBM * kBK; i += kThreads) {
      const int64_t r = m0 + i / kBK, k = k0 + i % kBK;
      sA[i % kBK][i / kBK] = r < p.M && k < p.K ? e4m3_to_f(p.a[r * p.lda + k]) : 0.f;
    }
    for (int i = threadIdx.x; i < kBN * kBK; i += kThreads) {
      const int64_t r = n0 + i / kBK, k = k0 + i % kBK;
      sB[i % kBK][i / kBK] = r < p.N && k < p.K ? e4m3_to_f(p.b[r * p.ldb + k]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kBK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] += sA[k][ty * 4 + i] * sB[k][tx * 4 + j];
    __syncthreads();
    if (k0 % 128 == 128 - kBK || k0 + kBK >= p.K) {  // a k-block is complete
      const int64_t kb = k0 / 128;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
          if (m < p.M && n < p.N)
            acc[i][j] += part[i][j] * (p.sa[kb * p.ld_sa + m] *
                                       (p.b_block ? p.sb[n / 128 * p.ld_sb + kb]
                                                  : p.sb[kb * p.ld_sb + n]));
          part[i][j] = 0.f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.M || n >= p.N) continue;
      if (p.c_fp32) static_cast<float*>(p.c)[m * p.ldc + n] = acc[i][j];
      else static_cast<__nv_bfloat16*>(p.c)[m * p.ldc + n] = __float2bfloat16_rn(acc[i][j]);
    }
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status_t fp8_block_gemm(const uint8_t* a, int64_t lda, const float* sa,
                                       int64_t ld_sa, const uint8_t* b, int64_t ldb,
                                       const float* sb, int64_t ld_sb, int32_t b_scale, void* c,
                                       int64_t ldc, int32_t c_dtype, int64_t M, int64_t N,
                                       int64_t K, int32_t* err, moe_stream_t stream) {
  if (M < 0 || N < 0 || K < 1) return fail(MOE_ERR_INVALID_ARG, "M, N must be >= 0 and K >= 1");
  const int64_t most = (int64_t)INT32_MAX - 256;
  if (M > most || N > most || K > most) return fail(MOE_ERR_UNSUPPORTED, "M, N or K too large");
  if (b_scale != 0 && b_scale != 1) return fail(MOE_ERR_INVALID_ARG, "b_scale must be 0 or 1");
  if (c_dtype != MOE_DT_BF16 && c_dtype != MOE_DT_FP32)
    return fail(MOE_ERR_INVALID_ARG, "unknown dtype %d", c_dtype);
  const int64_t kb = (K + 127) / 128;
  if (lda < K || ldb < K || ldc < N || ld_sa < M || ld_sb < (b_scale ? kb : N))
    return fail(MOE_ERR_INVALID_ARG, "a row stride is smaller than its row");
  if (M == 0 || N == 0) return MOE_OK;
  if (!a || !b || !sa || !sb || !c) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  auto at = [](const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; };
  if (!at(a, 16) || !at(b, 16) || lda % 16 || ldb % 16)
    return fail(MOE_ERR_INVALID_ARG, "a and b must be 16-byte aligned with strides of 16 bytes");
  if (!at(sa, 16) || ld_sa % 4 || !at(sb, b_scale ? 4 : 16) || (!b_scale && ld_sb % 4))
    return fail(MOE_ERR_INVALID_ARG,
                "1 x 128 scales must be 16-byte aligned with a stride of a multiple of 4");
  if (!at(c, c_dtype == MOE_DT_FP32 ? 4 : 2) || !at(err, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  Fp8Args p = {a, b, lda, ldb, sa, sb, ld_sa, ld_sb, b_scale, c, ldc, c_dtype == MOE_DT_FP32,
               M, N, K};
  if ((M + kBM - 1) / kBM > 65535) return fail(MOE_ERR_UNSUPPORTED, "M too large");
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  fp8_gemm_plain_kernel<<<dim3((unsigned)((N + kBN - 1) / kBN), (unsigned)((M + kBM - 1) / kBM)),
                          kThreads, 0, s>>>(p);
  count_launch(s, MOE_K_FP8_GEMM);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_fail(e, "fp8 gemm launch");
  return MOE_OK;
}
