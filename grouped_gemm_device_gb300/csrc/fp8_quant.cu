// E4M3 quantisers with one fp32 scale for each block of 128: blocks of 1 x 128 along the rows
// and, transposed, along the columns (fp8_block_quantize_rows), and blocks of 128 x 128 with the
// codes in both orders (fp8_block_quantize_weight); include/moegmm.h has the definition.
//
// Bound by HBM: 2 bytes read and 1 byte written an element and copy. A block takes a 128 x 128
// tile, so that every scale it needs, in either direction, is a maximum over values it holds, and
// reads the input once for both copies. A thread holds 8 rows x 8 columns: a row's 8 codes are
// one 8-byte store, a column's 8 codes one 8-byte store into a transposed tile in shared memory.
#include "kernels.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr int kPitch = kTile + 16;  // transposed tile: 16-byte rows stay aligned
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100
constexpr float kE4M3Max = 448.0f;

// max with NaN ignored on purpose: a NaN value keeps its own NaN code
MOE_DEVICE float amax_of(float m, float v) { return fmaxf(m, fabsf(v)); }
MOE_DEVICE float scale_of(float amax) { return fmaxf(amax, kTiny) / kE4M3Max; }
MOE_DEVICE float factor_of(float amax) { return kE4M3Max / fmaxf(amax, kTiny); }

struct QuantArgs {
  const uint16_t* x;
  int64_t ldx, M, N;
  uint8_t* q;        // codes as x lies, row stride ldq
  int64_t ldq;
  float* s;          // ROWS: [ceil(N/128), M] stride lds; SQUARE: [ceil(M/128), ceil(N/128)]
  int64_t lds;
  uint8_t* qt;       // codes transposed [N, M], row stride ldqt
  int64_t ldqt;
  float* st;         // ROWS: [ceil(M/128), N] stride ldst; SQUARE: [ceil(N/128), ceil(M/128)]
  int64_t ldst;
  int vec_in, vec_q, vec_qt;  // 16-byte loads, 8-byte and 16-byte stores are aligned
  int64_t tiles_n, tiles;
};

template <bool ROW, bool COL, bool SQUARE>
__global__ void __launch_bounds__(kThreads) fp8_quantize_kernel(const QuantArgs a) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float s_max[8][kTile];
  __shared__ __align__(16) uint8_t s_t[COL ? kTile * kPitch : 16];
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // column and row group of 8
  const int warp = threadIdx.x >> 5;
  for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const int64_t tm = tile / a.tiles_n, tn = tile % a.tiles_n;
    const int64_t r0 = tm * kTile + rg * 8, c0 = tn * kTile + cg * 8;
    float v[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint16_t* p = a.x + (r0 + i) * a.ldx + c0;
      if (a.vec_in && r0 + i < a.M && c0 + 8 <= a.N) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[i][2 * j] = bf16_lo(u[j]);
          v[i][2 * j + 1] = bf16_hi(u[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          v[i][j] = r0 + i < a.M && c0 + j < a.N
                        ? __uint_as_float((uint32_t)p[j] << 16) : 0.f;
      }
    }
    float fr[8], fc[8];  // factor of each row and of each column of this thread
    if constexpr (SQUARE) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = amax_of(m, v[i][j]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      __syncthreads();  // the previous tile's readers are done
      if ((threadIdx.x & 31) == 0) s_max[0][warp] = m;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) m = fmaxf(m, s_max[0][w]);
      if (threadIdx.x == 0) {
        a.s[tm * a.lds + tn] = scale_of(m);
        if (COL) a.st[tn * a.ldst + tm] = scale_of(m);
      }
      const float f = factor_of(m);
#pragma unroll
      for (int i = 0; i < 8; ++i) fr[i] = fc[i] = f;
    } else {
      if constexpr (ROW) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float m = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) m = amax_of(m, v[i][j]);
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
          fr[i] = factor_of(m);
          if (cg == i && r0 + i < a.M) a.s[tn * a.lds + r0 + i] = scale_of(m);
        }
      }
      if constexpr (COL) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float m = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) m = amax_of(m, v[i][j]);
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
          if ((threadIdx.x & 16) == 0) s_max[warp][cg * 8 + j] = m;
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float m = 0.f;
#pragma unroll
          for (int w = 0; w < 8; ++w) m = fmaxf(m, s_max[w][cg * 8 + j]);
          fc[j] = factor_of(m);
          if (rg == j && c0 + j < a.N) a.st[tm * a.ldst + c0 + j] = scale_of(m);
        }
      }
    }
    if constexpr (ROW) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (r0 + i >= a.M || c0 >= a.N) continue;
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = cvt_e4m3x2(v[i][4 * h] * fr[i], v[i][4 * h + 1] * fr[i]) |
                 (cvt_e4m3x2(v[i][4 * h + 2] * fr[i], v[i][4 * h + 3] * fr[i]) << 16);
        uint8_t* q = a.q + (r0 + i) * a.ldq + c0;
        if (a.vec_q && c0 + 8 <= a.N) {
          *reinterpret_cast<uint2*>(q) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c0 + j < a.N) q[j] = (uint8_t)(w[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
    if constexpr (COL) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = cvt_e4m3x2(v[4 * h][j] * fc[j], v[4 * h + 1][j] * fc[j]) |
                 (cvt_e4m3x2(v[4 * h + 2][j] * fc[j], v[4 * h + 3][j] * fc[j]) << 16);
        *reinterpret_cast<uint2*>(&s_t[(cg * 8 + j) * kPitch + rg * 8]) = make_uint2(w[0], w[1]);
      }
      __syncthreads();
      // 128 transposed rows of 128 bytes, eight 16-byte pieces each
      for (int p = threadIdx.x; p < kTile * 8; p += kThreads) {
        const int64_t c = tn * kTile + (p >> 3), r = tm * kTile + (p & 7) * 16;
        if (c >= a.N || r >= a.M) continue;
        const uint8_t* src = &s_t[(p >> 3) * kPitch + (p & 7) * 16];
        uint8_t* dst = a.qt + c * a.ldqt + r;
        if (a.vec_qt && r + 16 <= a.M) {
          *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(src);
        } else {
          for (int j = 0; j < 16 && r + j < a.M; ++j) dst[j] = src[j];
        }
      }
      __syncthreads();
    }
  }
}

template <bool ROW, bool COL, bool SQUARE>
cudaError_t launch_quant(const QuantArgs& a, cudaStream_t s) {
  const int64_t most = (int64_t)std::max(device_sms(), 1) * 16;
  fp8_quantize_kernel<ROW, COL, SQUARE><<<(unsigned)std::min(a.tiles, most), kThreads, 0, s>>>(a);
  count_launch(s, MOE_K_FP8_QUANTIZE);
  return cudaGetLastError();
}

bool aligned_to(const void* p, int64_t ld, int bytes) {
  return (reinterpret_cast<uintptr_t>(p) % bytes) == 0 && ld % bytes == 0;
}

void set_input(QuantArgs& a, const void* x, int64_t ldx, int64_t M, int64_t N) {
  a.x = static_cast<const uint16_t*>(x);
  a.ldx = ldx;
  a.M = M;
  a.N = N;
  a.tiles_n = (N + kTile - 1) / kTile;
  a.tiles = a.tiles_n * ((M + kTile - 1) / kTile);
  a.vec_in = aligned_to(x, ldx * 2, 16);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t fp8_block_quantize_rows(const void* x, int64_t ldx, int64_t M, int64_t N,
                                     uint8_t* q_row, int64_t ld_qrow, float* s_row,
                                     int64_t ld_srow, uint8_t* q_col, int64_t ld_qcol,
                                     float* s_col, int64_t ld_scol, moe_stream_t stream) {
  const bool row = q_row || s_row, col = q_col || s_col;
  if (M < 0 || N < 0) return fail(MOE_ERR_INVALID_ARG, "negative size");
  if (M > INT32_MAX || N > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "M or N too large");
  if (!row && !col) return fail(MOE_ERR_INVALID_ARG, "neither copy requested");
  if ((row && (!q_row || !s_row)) || (col && (!q_col || !s_col)))
    return fail(MOE_ERR_INVALID_ARG, "a copy needs both its codes and its scales");
  if (ldx < N || (row && (ld_qrow < N || ld_srow < M)) || (col && (ld_qcol < M || ld_scol < N)))
    return fail(MOE_ERR_INVALID_ARG, "a row stride is smaller than its row");
  if (M == 0 || N == 0) return MOE_OK;
  if (!x || (reinterpret_cast<uintptr_t>(x) & 1) || (reinterpret_cast<uintptr_t>(s_row) & 3) ||
      (reinterpret_cast<uintptr_t>(s_col) & 3))
    return fail(MOE_ERR_INVALID_ARG, "x must be non-NULL, tensors aligned to their elements");
  QuantArgs a = {};
  set_input(a, x, ldx, M, N);
  a.q = q_row; a.ldq = ld_qrow; a.s = s_row; a.lds = ld_srow;
  a.qt = q_col; a.ldqt = ld_qcol; a.st = s_col; a.ldst = ld_scol;
  a.vec_q = aligned_to(q_row, ld_qrow, 8);
  a.vec_qt = aligned_to(q_col, ld_qcol, 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = row && col ? launch_quant<true, true, false>(a, s)
                  : row      ? launch_quant<true, false, false>(a, s)
                             : launch_quant<false, true, false>(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 quantiser launch");
  return MOE_OK;
}

moe_status_t fp8_block_quantize_weight(const void* w, int64_t ldw, int64_t N, int64_t K,
                                       uint8_t* q, int64_t ldq, float* sc, uint8_t* qt,
                                       int64_t ldqt, float* st, moe_stream_t stream) {
  if (N < 0 || K < 0) return fail(MOE_ERR_INVALID_ARG, "negative size");
  if (N > INT32_MAX || K > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "N or K too large");
  if ((qt != nullptr) != (st != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "qt and st go together");
  if (ldw < K || ldq < K || (qt && ldqt < N))
    return fail(MOE_ERR_INVALID_ARG, "a row stride is smaller than its row");
  if (N == 0 || K == 0) return MOE_OK;
  if (!w || !q || !sc) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  if ((reinterpret_cast<uintptr_t>(w) & 1) || (reinterpret_cast<uintptr_t>(sc) & 3) ||
      (reinterpret_cast<uintptr_t>(st) & 3))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  QuantArgs a = {};
  set_input(a, w, ldw, N, K);
  a.q = q; a.ldq = ldq; a.s = sc; a.lds = a.tiles_n;
  a.qt = qt; a.ldqt = ldqt; a.st = st; a.ldst = (N + kTile - 1) / kTile;
  a.vec_q = aligned_to(q, ldq, 8);
  a.vec_qt = aligned_to(qt, ldqt, 16);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = qt ? launch_quant<true, true, true>(a, s) : launch_quant<true, false, true>(a, s);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 weight quantiser launch");
  return MOE_OK;
}

}  // extern "C"
