// E4M3 quantisers with one fp32 scale for each block of 128: blocks of 1 x 128 along the rows
// and, transposed, along the columns (fp8_block_quantize_rows), and blocks of 128 x 128 with the
// codes in both orders (fp8_block_quantize_weight); include/moegmm.h has the definition.
//
// Bound by HBM: 2 bytes read and 1 byte written an element and copy. Rows alone stream: eight lanes
// hold a block. Anything with columns takes 128 x 128 tiles, so that every scale it needs, in
// either direction, is a maximum over values the thread block holds and one read of the input
// serves both copies. Rows alone: 8192 x 14336 53 us (6.7 TB/s, all of the measured copy rate);
// both copies: 95 us (5.0 TB/s; the tile's barriers and its pass through shared memory); weights of
// 14336 x 4096, both orders: 42 us (5.6 TB/s); one row of 7168: 1.7 us. Maxima are taken on the
// bf16 values themselves (a maximum rounds nothing), two at a time.
#include "kernels.cuh"
#include "realign.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100
constexpr float kE4M3Max = 448.0f;

MOE_DEVICE float scale_of(float amax) { return fmaxf(amax, kTiny) / kE4M3Max; }
MOE_DEVICE float factor_of(float amax) { return kE4M3Max / fmaxf(amax, kTiny); }
// Two bf16 maxima at once. A NaN loses to a number on purpose: it keeps its own NaN code and
// leaves its block's scale alone.
MOE_DEVICE uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
MOE_DEVICE uint32_t abs2(uint32_t a) { return a & 0x7FFF7FFFu; }
MOE_DEVICE uint32_t max2_halves(uint32_t a) { return max2(a, (a >> 16) | (a << 16)); }

// Four codes of two packed pairs.
MOE_DEVICE uint32_t codes4(uint32_t a, uint32_t b, float f) {
  return cvt_e4m3x2(bf16_lo(a) * f, bf16_hi(a) * f) |
         (cvt_e4m3x2(bf16_lo(b) * f, bf16_hi(b) * f) << 16);
}

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
  int vec_in, vec_q, vec_qt;  // 16-byte loads, 8-byte (rows alone: 16) and 16-byte stores
  int64_t tiles_n, tiles;
};

// 8 consecutive values of a row from column c (zeros past column N).
MOE_DEVICE uint4 load8(const uint16_t* row, int64_t c, int64_t N, bool vec) {
  if (vec && c + 8 <= N) return *reinterpret_cast<const uint4*>(row + c);
  return c < N ? load16_any(row + c, (N - c) * 2) : make_uint4(0, 0, 0, 0);
}

// Rows alone: a warp takes 512 columns (16 a lane, eight lanes a block) of kRows rows.
constexpr int kRows = 4;
constexpr unsigned kFewBlocks = 64;
__global__ void __launch_bounds__(kThreads) fp8_quantize_rows_kernel(const QuantArgs a) {
  MOE_GRIDDEP_ENTRY();
  // a few rows: the product that follows may set itself up meanwhile (with many, its CTAs would
  // take shared memory from blocks still to come)
  if (gridDim.x <= kFewBlocks) griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t segs = (a.N + 511) / 512, groups = (a.M + kRows - 1) / kRows;
  const int64_t step = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); u < segs * groups;
       u += step) {
    const int64_t r0 = (u % groups) * kRows, c = (u / groups) * 512 + lane * 16;
    uint4 w[kRows][2];
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[i][h] = r0 + i < a.M ? load8(a.x + (r0 + i) * a.ldx, c + 8 * h, a.N, a.vec_in)
                               : make_uint4(0, 0, 0, 0);
    uint32_t m[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const uint4 &p = w[i][0], &q = w[i][1];
      m[i] = max2(max2(max2(abs2(p.x), abs2(p.y)), max2(abs2(p.z), abs2(p.w))),
                  max2(max2(abs2(q.x), abs2(q.y)), max2(abs2(q.z), abs2(q.w))));
    }
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < kRows; ++i) m[i] = max2(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], o));
    float amax[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) amax[i] = bf16_lo(max2_halves(m[i]));
    // lane i of a block's eight writes row i's scale (its own columns may lie past the end)
    if ((lane & 7) < kRows && (c & ~(int64_t)127) < a.N) {
      float v = amax[0];
#pragma unroll
      for (int i = 1; i < kRows; ++i)
        if ((lane & 7) == i) v = amax[i];
      if (r0 + (lane & 7) < a.M) a.s[(c >> 7) * a.lds + r0 + (lane & 7)] = scale_of(v);
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (r0 + i >= a.M || c >= a.N) continue;
      const float f = factor_of(amax[i]);
      const uint4 &p = w[i][0], &q = w[i][1];
      const uint4 o = make_uint4(codes4(p.x, p.y, f), codes4(p.z, p.w, f), codes4(q.x, q.y, f),
                                 codes4(q.z, q.w, f));
      uint8_t* d = a.q + (r0 + i) * a.ldq + c;
      if (a.vec_q && c + 16 <= a.N) {
        *reinterpret_cast<uint4*>(d) = o;
      } else {
        const uint32_t ow[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < a.N) d[j] = (uint8_t)(ow[j >> 2] >> (8 * (j & 3)));
      }
    }
  }
}

// Tiles of 128 x 128. Thread (rg, cg) holds rows 8 rg.. and columns 8 cg.. as packed bf16; a
// row's 8 codes are one 8-byte store, a column's 8 codes one 8-byte store into the transposed
// tile in shared memory, whose 16-byte pieces are XOR-rotated by the row's column group so that
// a warp's stores and the row-wise reads touch all banks.
template <bool ROW, bool COL, bool SQUARE>
__global__ void __launch_bounds__(kThreads, 3) fp8_quantize_kernel(const QuantArgs a) {
  MOE_GRIDDEP_ENTRY();
  __shared__ uint32_t s_max[8][4][16];  // each warp's column maxima, two a word
  __shared__ __align__(16) float s_fc[4][16][2];
  __shared__ __align__(16) uint8_t s_t[COL ? kTile * kTile : 16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int cg = threadIdx.x & 15, rg = threadIdx.x >> 4;  // column and row group of 8
  for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
    const int64_t tm = tile / a.tiles_n, tn = tile % a.tiles_n;
    const int64_t r0 = tm * kTile + rg * 8, c0 = tn * kTile + cg * 8;
    uint32_t w[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint4 v = r0 + i < a.M ? load8(a.x + (r0 + i) * a.ldx, c0, a.N, a.vec_in)
                                   : make_uint4(0, 0, 0, 0);
      w[i][0] = v.x;
      w[i][1] = v.y;
      w[i][2] = v.z;
      w[i][3] = v.w;
    }
    uint32_t mc[4];  // column maxima of this thread's 8 rows
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mc[j] = abs2(w[0][j]);
#pragma unroll
      for (int i = 1; i < 8; ++i) mc[j] = max2(mc[j], abs2(w[i][j]));
    }
    float fr = 0.f;  // ROW: factor of row (lane & 7) of this row group; SQUARE: the tile's
    if constexpr (SQUARE) {
      uint32_t m = max2(max2(mc[0], mc[1]), max2(mc[2], mc[3]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max2(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (lane == 0) s_max[0][0][warp] = m;  // free: the last tile's barriers came after its reads
      __syncthreads();
#pragma unroll
      for (int v = 0; v < 8; ++v) m = max2(m, s_max[0][0][v]);
      const float amax = bf16_lo(max2_halves(m));
      if (threadIdx.x == 0) {
        a.s[tm * a.lds + tn] = scale_of(amax);
        if (COL) a.st[tn * a.ldst + tm] = scale_of(amax);
      }
      fr = factor_of(amax);
      if (!COL) __syncthreads();  // s_max is written again in the next tile
    } else {
      // rows 2i and 2i + 1 in one word, over the row group's 16 lanes
      uint32_t mr[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t m2[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t* v = w[2 * i + h];
          m2[h] = max2_halves(max2(max2(abs2(v[0]), abs2(v[1])), max2(abs2(v[2]), abs2(v[3]))));
        }
        mr[i] = (m2[0] & 0xFFFFu) | (m2[1] << 16);
      }
      if constexpr (ROW) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
#pragma unroll
          for (int i = 0; i < 4; ++i) mr[i] = max2(mr[i], __shfl_xor_sync(0xFFFFFFFFu, mr[i], o));
        uint32_t m = mr[0];
#pragma unroll
        for (int i = 1; i < 4; ++i)
          if (((lane & 7) >> 1) == i) m = mr[i];
        const float amax = (lane & 1) ? bf16_hi(m) : bf16_lo(m);
        fr = factor_of(amax);
        if ((lane & 8) == 0 && r0 + (lane & 7) < a.M)
          a.s[tn * a.lds + r0 + (lane & 7)] = scale_of(amax);
      }
      if constexpr (COL) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          mc[j] = max2(mc[j], __shfl_xor_sync(0xFFFFFFFFu, mc[j], 16));
          if (lane < 16) s_max[warp][j][cg] = mc[j];
        }
        __syncthreads();
        if (threadIdx.x < 64) {  // columns 2 * (4 * cg + j) and the next
          const int j = threadIdx.x >> 4;
          uint32_t m = s_max[0][j][cg];
#pragma unroll
          for (int v = 1; v < 8; ++v) m = max2(m, s_max[v][j][cg]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float amax = h ? bf16_hi(m) : bf16_lo(m);
            const int64_t col = tn * kTile + cg * 8 + 2 * j + h;
            s_fc[j][cg][h] = factor_of(amax);
            if (col < a.N) a.st[tm * a.ldst + col] = scale_of(amax);
          }
        }
        __syncthreads();
      }
    }
    if constexpr (ROW) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float f = SQUARE ? fr : __shfl_sync(0xFFFFFFFFu, fr, (lane & 16) | i);
        if (r0 + i >= a.M || c0 >= a.N) continue;
        const uint32_t o[2] = {codes4(w[i][0], w[i][1], f), codes4(w[i][2], w[i][3], f)};
        uint8_t* q = a.q + (r0 + i) * a.ldq + c0;
        if (a.vec_q && c0 + 8 <= a.N) {
          *reinterpret_cast<uint2*>(q) = make_uint2(o[0], o[1]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c0 + j < a.N) q[j] = (uint8_t)(o[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
    if constexpr (COL) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[2] = {fr, fr};
        if (!SQUARE) {
          const float2 v = *reinterpret_cast<const float2*>(s_fc[j][cg]);
          f[0] = v.x;
          f[1] = v.y;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[2];
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            float v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t x = w[4 * g + i][j];
              v[i] = (h ? bf16_hi(x) : bf16_lo(x)) * f[h];
            }
            o[g] = cvt_e4m3x2(v[0], v[1]) | (cvt_e4m3x2(v[2], v[3]) << 16);
          }
          const int row = cg * 8 + 2 * j + h, piece = (rg >> 1) ^ (cg & 7);
          *reinterpret_cast<uint2*>(&s_t[row * kTile + piece * 16 + (rg & 1) * 8]) =
              make_uint2(o[0], o[1]);
        }
      }
      __syncthreads();
      // 128 transposed rows of 128 bytes, eight 16-byte pieces each
#pragma unroll
      for (int p = threadIdx.x; p < kTile * 8; p += kThreads) {
        const int row = p >> 3, piece = p & 7;
        const int64_t c = tn * kTile + row, r = tm * kTile + piece * 16;
        if (c >= a.N || r >= a.M) continue;
        const uint8_t* src = &s_t[row * kTile + ((piece ^ ((row >> 3) & 7)) * 16)];
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
  cudaError_t e = launch_pdl(fp8_quantize_kernel<ROW, COL, SQUARE>,
                             (unsigned)std::min(a.tiles, most), kThreads, 0, s, 1, a);
  count_launch(s, MOE_K_FP8_QUANTIZE);
  return e;
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
  if (row && !col) {
    a.vec_q = aligned_to(q_row, ld_qrow, 16);
    const int64_t warps = (N + 511) / 512 * ((M + kRows - 1) / kRows);
    const int64_t most = (int64_t)std::max(device_sms(), 1) * 32;
    const int64_t blocks = std::min((warps + kThreads / 32 - 1) / (kThreads / 32), most);
    cudaError_t e =
        launch_pdl(fp8_quantize_rows_kernel, (unsigned)blocks, kThreads, 0, s, 1, a);
    count_launch(s, MOE_K_FP8_QUANTIZE);
    if (e != cudaSuccess) return cuda_fail(e, "fp8 quantiser launch");
    return MOE_OK;
  }
  cudaError_t e =
      row ? launch_quant<true, true, false>(a, s) : launch_quant<false, true, false>(a, s);
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
