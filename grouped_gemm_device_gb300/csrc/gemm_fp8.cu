// Dense product of E4M3 operands with an fp32 scale for each block of 128 (fp8_block_gemm in
// include/moegmm.h):
//
//   C[m][n] = sum over k-blocks b of sa[b][m] * sb * (a[m, b] . b[n, b])
//
// The scales are arbitrary fp32 numbers, so the tensor cores cannot apply them (their block-scaled
// forms take powers of two or E4M3 scales over 16 or 32 values): each 128-element k-block is one
// unscaled product in TMEM, and the epilogue warps add it, scaled, to fp32 sums in registers while
// the tensor cores work on the next one in another TMEM buffer.
//
// One CTA: warp 0 loads (TMA, K-major 128-byte-swizzled boxes of 128 bytes; the 1 x 128 scales of
// a k-block as one row of their [k-block, row] matrix), warp 1 issues the MMAs (128 x BN x 32,
// kind::f8f6f4), warps 2-9 hold the 128 x BN fp32 sums (warp w: TMEM lanes 32 (w % 4).., half of
// the columns). P is the operand on the 128-row side, Q the one on the BN-column side.
//   Many rows: P = a, Q = b, tiles of 128 x 256; a result row is contiguous in a thread.
//   Few rows (M <= 128): P = b, Q = a (BN = M rounded up), so that the whole 128-row side is
//   filled with features and the small operand costs what it holds; the result is written
//   transposed, one feature a lane.
//   Few tiles: the k-blocks are split over a cluster of 2-8 CTAs, whose sums are added through
//   distributed shared memory in the order of their ranks.
#include "gemm_common.cuh"

namespace moe {
namespace {

constexpr int BM = 128;
constexpr int BK = 128;              // E4M3 elements (bytes) per k-block
constexpr int MMA_K = 32;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxStages = 8;
constexpr int kMaxSlots = 12;
constexpr int kMaxSplit = 8;

struct Fp8Args {
  CUtensorMap tmP, tmQ;    // codes [rows, K]
  CUtensorMap tmSP, tmSQ;  // 1 x 128 scales [k-blocks, rows] (those that are vectors)
  const float* sp;         // 128 x 128 scales of P, [ceil(rows/128), k-blocks] (sp_vec = 0)
  const float* sq;         // the same of Q (QV = 0)
  int64_t ld_sp, ld_sq;
  int sp_vec;
  int swapped;             // P = b, Q = a: C[q][p]
  void* c;
  int64_t ldc;
  int c_fp32;
  int align;               // bytes every row of C is aligned to (16 or 32), or 0
  int rows_p, rows_q, K;
  int tiles_p, tiles_q;
  int split;               // CTAs of a cluster that share one tile's k-blocks
  int* err;
};

template <int BN>
struct Smem {
  static constexpr int P_BYTES = BM * BK;
  static constexpr int Q_BYTES = BN * BK;
  static constexpr int STAGE = P_BYTES + Q_BYTES;
  static constexpr int STAGES = BN >= 256 ? 4 : BN >= 128 ? 6 : 8;
  static constexpr int BUFS = BN >= 256 ? 2 : 4;       // TMEM accumulators
  static constexpr int TMEM_COLS = BUFS * BN;          // 64 .. 512, a power of two
  static constexpr int SLOTS = STAGES + BUFS;          // scale rows in flight
  static constexpr int SP_BYTES = BM * 4;
  static constexpr int SQ_BYTES = BN * 4 < 128 ? 128 : BN * 4;
  static constexpr int SLOT = SP_BYTES + SQ_BYTES;
  static constexpr int SLOT_OFF = STAGES * STAGE;
  static constexpr int CTRL_OFF = SLOT_OFF + SLOTS * SLOT;
  static constexpr int TOTAL = CTRL_OFF + 512 + 1024;
  static_assert(TOTAL <= 232448, "shared memory above the per-block limit");
  static_assert(STAGES <= kMaxStages && SLOTS <= kMaxSlots, "control block");
  static_assert(STAGES * STAGE >= BM * BN * 4, "the split sums fit in the stages");
};

struct Ctrl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t sfull[kMaxSlots], sempty[kMaxSlots];
  uint64_t tfull[4], tempty[4];
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
};
static_assert(sizeof(Ctrl) <= 512, "control block");

// D[tmem] (+)= A[smem] * B[smem]^T, kind::f8f6f4, fp32 accumulation.
MOE_DEVICE void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// fp32 accumulator (bit 4), E4M3 A and B (format 0), both K-major.
constexpr uint32_t idesc_f8(int M, int N) {
  return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// Two fp32 lanes at a time: acc += {lo, hi} * f, and a * b.
MOE_DEVICE void fma2(uint64_t& acc, uint32_t lo, uint32_t hi, uint64_t f) {
  asm("{\n\t.reg .b64 t;\n\tmov.b64 t, {%1, %2};\n\tfma.rn.f32x2 %0, t, %3, %0;\n\t}"
      : "+l"(acc)
      : "r"(lo), "r"(hi), "l"(f));
}
MOE_DEVICE uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
MOE_DEVICE uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
MOE_DEVICE float lo_of(uint64_t v) { return __uint_as_float((uint32_t)v); }
MOE_DEVICE float hi_of(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// W consecutive TMEM columns of this warp's 32 lanes.
template <int W>
MOE_DEVICE void tmem_ld(uint32_t taddr, uint32_t (&r)[W]) {
  if constexpr (W == 32) tmem_ld_32x32b_x32(taddr, r);
  else if constexpr (W == 16) tmem_ld_32x32b_x16(taddr, r);
  else tmem_ld_32x32b_x8(taddr, r);
}

MOE_DEVICE float ld_shared_cluster(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

// n (a multiple of 8, at most 32 here per step) consecutive results of one row.
template <int W>
MOE_DEVICE void store_row(const Fp8Args& p, int64_t row, int col, const float (&v)[W]) {
  if (p.c_fp32) {
    float* o = static_cast<float*>(p.c) + row * p.ldc + col;
    if (p.align && col + W <= p.rows_q) {
#pragma unroll
      for (int i = 0; i < W; i += 8) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[i + j]);
        if (p.align == 32) {
          st_global_v8(o + i, w);
        } else {
          reinterpret_cast<uint4*>(o + i)[0] = make_uint4(w[0], w[1], w[2], w[3]);
          reinterpret_cast<uint4*>(o + i)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col + i < p.rows_q) o[i] = v[i];
    }
  } else {
    __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.c) + row * p.ldc + col;
    if (p.align && col + W <= p.rows_q) {
#pragma unroll
      for (int i = 0; i < W; i += 16) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < (W < 16 ? 4 : 8); ++j)
          w[j] = pack_bf16x2(v[i + 2 * j], v[i + 2 * j + 1]);
        if (W >= 16 && p.align == 32) {
          st_global_v8(o + i, w);
        } else {
          reinterpret_cast<uint4*>(o + i)[0] = make_uint4(w[0], w[1], w[2], w[3]);
          if (W >= 16) reinterpret_cast<uint4*>(o + i)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (col + i < p.rows_q) o[i] = __float2bfloat16_rn(v[i]);
    }
  }
}
// One result of the swapped form: row `prow` of P, row `qrow` of Q.
MOE_DEVICE void store_swapped(const Fp8Args& p, int prow, int64_t qrow, float v) {
  if (p.c_fp32) static_cast<float*>(p.c)[qrow * p.ldc + prow] = v;
  else static_cast<__nv_bfloat16*>(p.c)[qrow * p.ldc + prow] = __float2bfloat16_rn(v);
}

template <int BN, bool QV>
__global__ void __launch_bounds__(kThreads, 1) fp8_gemm_kernel(const __grid_constant__ Fp8Args p) {
  MOE_GRIDDEP_ENTRY();
  using L = Smem<BN>;
  constexpr int STAGES = L::STAGES, BUFS = L::BUFS, SLOTS = L::SLOTS;
  constexpr int CW = BN / 2;                  // columns a warp holds
  constexpr int CH = CW < 32 ? CW : 32;       // columns a TMEM load
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  Ctrl& c = *reinterpret_cast<Ctrl*>(smem + L::CTRL_OFF);
  volatile int* abort = &c.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;
  const int total = p.tiles_p * p.tiles_q;
  const int tile0 = (int)blockIdx.x / p.split, tstep = (int)gridDim.x / p.split;
  const int nkb_all = (p.K + BK - 1) / BK;
  const int kb0 = (int)((int64_t)nkb_all * rank / p.split);
  const int kb1 = (int)((int64_t)nkb_all * (rank + 1) / p.split);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&c.full[s], 1);
      mbar_init(&c.empty[s], 1);
    }
    for (int s = 0; s < SLOTS; ++s) {
      mbar_init(&c.sfull[s], 1);
      mbar_init(&c.sempty[s], kEpiWarps);
    }
    for (int s = 0; s < BUFS; ++s) {
      mbar_init(&c.tfull[s], 1);
      mbar_init(&c.tempty[s], kEpiWarps);
    }
    mbar_init(&c.drain, 1);
    fence_mbar_init();
    c.abort = 0;
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&p.tmP);
    tma_prefetch_desc(&p.tmQ);
  }
  if (warp == 1) {
    tmem_alloc(&c.tmem_base, L::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = c.tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      const uint32_t slot_tx = (p.sp_vec ? L::SP_BYTES : 0) + (QV ? BN * 4 : 0);
      int stage = 0, slot = 0;
      uint32_t phase = 0, sphase = 0;
      int64_t n_full = 0, n_slot = 0;  // loads armed so far
      bool ok = true;
      for (int tile = tile0; ok && tile < total; tile += tstep) {
        const int p0 = (tile % p.tiles_p) * BM, q0 = (tile / p.tiles_p) * BN;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&c.empty[stage], phase ^ 1, abort, p.err)) {
            ok = false;
            break;
          }
          uint8_t* sP = smem + stage * L::STAGE;
          mbar_arrive_expect_tx(&c.full[stage], L::STAGE);
          ++n_full;
          tma_load_2d(sP, &p.tmP, &c.full[stage], kb * BK, p0);
          tma_load_2d(sP + L::P_BYTES, &p.tmQ, &c.full[stage], kb * BK, q0);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
          if (slot_tx) {
            if (!mbar_wait(&c.sempty[slot], sphase ^ 1, abort, p.err)) {
              ok = false;
              break;
            }
            uint8_t* s = smem + L::SLOT_OFF + slot * L::SLOT;
            mbar_arrive_expect_tx(&c.sfull[slot], slot_tx);
            ++n_slot;
            if (p.sp_vec) tma_load_2d(s, &p.tmSP, &c.sfull[slot], p0, kb);
            if (QV) tma_load_2d(s + L::SP_BYTES, &p.tmSQ, &c.sfull[slot], q0, kb);
            if (++slot == SLOTS) {
              slot = 0;
              sphase ^= 1;
            }
          }
        }
      }
      // every load this thread issued lands before the CTA can exit: the last phase armed on
      // each barrier (load i of a ring of R sits at i % R with parity (i / R) & 1)
      const uint64_t t0 = globaltimer_ns();
      for (int64_t i = n_full > STAGES ? n_full - STAGES : 0; i < n_full; ++i)
        while (!mbar_try_wait(smem_u32(&c.full[i % STAGES]), (uint32_t)((i / STAGES) & 1)) &&
               globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      for (int64_t i = n_slot > SLOTS ? n_slot - SLOTS : 0; i < n_slot; ++i)
        while (!mbar_try_wait(smem_u32(&c.sfull[i % SLOTS]), (uint32_t)((i / SLOTS) & 1)) &&
               globaltimer_ns() - t0 < kWaitLimitNs) {
        }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true, issued = false;
      for (int tile = tile0; ok && tile < total; tile += tstep) {
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&c.tempty[buf], tphase ^ 1, abort, p.err) ||
              !mbar_wait(&c.full[stage], phase, abort, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sP = smem_u32(smem + stage * L::STAGE);
          const uint32_t sQ = sP + L::P_BYTES;
          const int rem = p.K - kb * BK;
          const int nsub = rem >= BK ? BK / MMA_K : (rem + MMA_K - 1) / MMA_K;
          for (int ks = 0; ks < nsub; ++ks)
            mma_f8_ss(tmem_base + buf * BN, smem_desc_sw128(sP + ks * MMA_K, 16, 1024),
                      smem_desc_sw128(sQ + ks * MMA_K, 16, 1024), idesc_f8(BM, BN), ks != 0);
          issued = true;
          mma_commit(&c.empty[stage]);
          mma_commit(&c.tfull[buf]);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
          if (++buf == BUFS) {
            buf = 0;
            tphase ^= 1;
          }
        }
      }
      if (issued) {
        mma_commit(&c.drain);
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&c.drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ epilogue warps
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int row = q * 32 + lane;  // of the tile's P side
    const bool slots = p.sp_vec || QV;
    int buf = 0, slot = 0;
    uint32_t tphase = 0, sphase = 0;
    bool ok = true;
    for (int tile = tile0; tile < total; tile += tstep) {
      __syncwarp();  // rows past the end left the last tile early
      const int p0 = (tile % p.tiles_p) * BM, q0 = (tile / p.tiles_p) * BN;
      uint64_t acc[CW / 2];
#pragma unroll
      for (int i = 0; i < CW / 2; ++i) acc[i] = 0;
      // 128 x 128 scales: one number a k-block for the whole tile side (a column half of a
      // 256-wide tile); a half past the last column reads the last block's and is never stored
      const float* spb = p.sp + (int64_t)(p0 >> 7) * p.ld_sp;
      const int qb = min((q0 + half * CW) >> 7, (p.rows_q - 1) >> 7);
      const float* sqb = QV ? nullptr : p.sq + (int64_t)qb * p.ld_sq;
      float sp_next = p.sp_vec ? 0.f : __ldg(spb + kb0);
      float sq_next = QV ? 0.f : __ldg(sqb + kb0);
      for (int kb = kb0; kb < kb1; ++kb) {
        float sp = sp_next, sq = sq_next;
        if (kb + 1 < kb1) {
          if (!p.sp_vec) sp_next = __ldg(spb + kb + 1);
          if (!QV) sq_next = __ldg(sqb + kb + 1);
        }
        const uint8_t* sl = smem + L::SLOT_OFF + slot * L::SLOT;
        // every give-up decision is warp-uniform (full-warp TMEM loads)
        bool got = true;
        if (slots) got = mbar_wait(&c.sfull[slot], sphase, abort, p.err);
        got = got && mbar_wait(&c.tfull[buf], tphase, abort, p.err);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (p.sp_vec) sp = reinterpret_cast<const float*>(sl)[row];
        const float* sqv = reinterpret_cast<const float*>(sl + L::SP_BYTES) + half * CW;
        const uint32_t taddr = tmem_base + buf * BN + half * CW + ((uint32_t)(q * 32) << 16);
        const uint64_t f = QV ? pack2(sp, sp) : pack2(sp * sq, sp * sq);
#pragma unroll
        for (int j = 0; j < CW / CH; ++j) {
          uint32_t r[CH];
          tmem_ld(taddr + j * CH, r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            uint64_t g = f;
            if (QV) g = mul2(f, *reinterpret_cast<const uint64_t*>(sqv + j * CH + 2 * i));
            fma2(acc[j * (CH / 2) + i], r[2 * i], r[2 * i + 1], g);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&c.tempty[buf]);
          if (slots) mbar_arrive(&c.sempty[slot]);
        }
        if (++buf == BUFS) {
          buf = 0;
          tphase ^= 1;
        }
        if (slots && ++slot == SLOTS) {
          slot = 0;
          sphase ^= 1;
        }
      }
      if (!ok) break;
      if (p.split > 1) {
        // this CTA's sums, column by column, where the stages were (every load has been used)
        float* st = reinterpret_cast<float*>(smem) + half * CW * BM + row;
#pragma unroll
        for (int i = 0; i < CW / 2; ++i) {
          st[(2 * i) * BM] = lo_of(acc[i]);
          st[(2 * i + 1) * BM] = hi_of(acc[i]);
        }
        break;  // one tile a cluster
      }
      if (p0 + row >= p.rows_p) continue;
      if (p.swapped) {
#pragma unroll
        for (int i = 0; i < CW; ++i) {
          const int64_t qr = q0 + half * CW + i;
          if (qr < p.rows_q)
            store_swapped(p, p0 + row, qr, i & 1 ? hi_of(acc[i / 2]) : lo_of(acc[i / 2]));
        }
      } else {
#pragma unroll
        for (int j = 0; j < CW / CH; ++j) {
          const int col = q0 + half * CW + j * CH;
          if (col >= p.rows_q) break;
          float v[CH];
#pragma unroll
          for (int i = 0; i < CH / 2; ++i) {
            v[2 * i] = lo_of(acc[j * (CH / 2) + i]);
            v[2 * i + 1] = hi_of(acc[j * (CH / 2) + i]);
          }
          store_row<CH>(p, p0 + row, col, v);
        }
      }
    }
  }

  if (p.split > 1) {
    // rank r adds columns [r BN / split, (r + 1) BN / split) of every CTA of the cluster, in the
    // order of the ranks, and stores them
    __syncthreads();
    cluster_sync_all();
    if (warp >= 2 && !*abort) {
      const int tid = threadIdx.x - 64;
      const int row = tid & 127, cg = tid >> 7;
      const int p0 = (tile0 % p.tiles_p) * BM, q0 = (tile0 / p.tiles_p) * BN;
      const int per = BN / p.split, c_lo = rank * per + cg * (per / 2);
      const uint32_t base = smem_u32(smem) + (uint32_t)row * 4;
      uint32_t peer[kMaxSplit];
#pragma unroll
      for (int s = 0; s < kMaxSplit; ++s)
        if (s < p.split) peer[s] = mapa_shared(base, (uint32_t)s);
      if (p0 + row < p.rows_p) {
        for (int i = c_lo; i < c_lo + per / 2; ++i) {
          const int64_t qr = q0 + i;
          if (qr >= p.rows_q) break;
          float v = 0.f;
#pragma unroll
          for (int s = 0; s < kMaxSplit; ++s)
            if (s < p.split) v += ld_shared_cluster(peer[s] + (uint32_t)i * (BM * 4));
          if (p.swapped) {
            store_swapped(p, p0 + row, qr, v);
          } else if (p.c_fp32) {
            static_cast<float*>(p.c)[(int64_t)(p0 + row) * p.ldc + qr] = v;
          } else {
            static_cast<__nv_bfloat16*>(p.c)[(int64_t)(p0 + row) * p.ldc + qr] =
                __float2bfloat16_rn(v);
          }
        }
      }
      __syncwarp();
    }
    // no CTA leaves while another may read its sums
    __syncthreads();
    cluster_sync_all();
  }
  griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, L::TMEM_COLS);
  }
}

// Codes [rows, K] with a row stride of ld bytes; one box is box_rows x 128 bytes.
bool tmap_codes(CUtensorMap* m, const uint8_t* q, int64_t rows, int64_t K, int64_t ld,
                uint32_t box_rows) {
  uint64_t dims[2] = {(uint64_t)K, (uint64_t)rows};
  uint64_t strides[1] = {(uint64_t)ld};
  uint32_t box[2] = {BK, box_rows};
  return make_tmap(m, q, 2, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_UINT8);
}
// Scales [k-blocks, rows] with a row stride of ld floats; one box is a row of `n` of them.
bool tmap_scales(CUtensorMap* m, const float* s, int64_t rows, int64_t kb, int64_t ld,
                 uint32_t n) {
  uint64_t dims[2] = {(uint64_t)rows, (uint64_t)kb};
  uint64_t strides[1] = {(uint64_t)ld * 4};
  uint32_t box[2] = {n, 1};
  return make_tmap(m, s, 2, dims, strides, box, CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                   CU_TENSOR_MAP_SWIZZLE_NONE);
}

struct Operand {
  const uint8_t* q;
  int64_t rows, ld;
  const float* s;
  int64_t ld_s;
  bool vec;
};

template <int BN, bool QV>
cudaError_t launch_gemm(Fp8Args& a, const Operand& P, const Operand& Q, cudaStream_t s) {
  const int64_t kb = (a.K + BK - 1) / BK;
  if (!tmap_codes(&a.tmP, P.q, P.rows, a.K, P.ld, BM) ||
      !tmap_codes(&a.tmQ, Q.q, Q.rows, a.K, Q.ld, BN) ||
      (P.vec && !tmap_scales(&a.tmSP, P.s, P.rows, kb, P.ld_s, BM)) ||
      (QV && !tmap_scales(&a.tmSQ, Q.s, Q.rows, kb, Q.ld_s, BN)))
    return cudaErrorInvalidValue;
  auto kern = fp8_gemm_kernel<BN, QV>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Smem<BN>::TOTAL);
  if (e != cudaSuccess) return e;
  const int tiles = a.tiles_p * a.tiles_q;
  const int sms = std::max(device_sms(), 1);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.split;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  const int grid = a.split > 1 ? tiles * a.split : std::min(tiles, sms);
  e = launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), Smem<BN>::TOTAL, s, attr,
                    a.split > 1 ? 1 : 0, a);
  count_launch(s, MOE_K_FP8_GEMM);
  return e;
}

struct Plan {
  int bn, split;
};

// Tile width and split of the k-blocks for P x Q rows, by the time of the longest-running SM in
// SM cycles: a k-block of a 128 x BN tile takes `kb_cycles` (its loads or its MMAs), a tile's
// results and first loads about 2000 on top, adding up a cluster's sums 1500.
Plan choose(int64_t rows_p, int64_t rows_q, int64_t nkb, bool swapped, int sms) {
  static const int widths[5] = {16, 32, 64, 128, 256};
  static const int kb_cycles[5] = {300, 310, 330, 380, 580};
  Plan best = {0, 1};
  int64_t best_t = INT64_MAX;
  const int64_t tp = (rows_p + BM - 1) / BM;
  for (int i = swapped ? 0 : 2; i < 5; ++i) {
    const int64_t tiles = tp * ((rows_q + widths[i] - 1) / widths[i]);
    for (int split = 1; split <= kMaxSplit; split *= 2) {
      if (split > 1 && (tiles * split > sms || split > nkb)) break;
      const int64_t waves = split > 1 ? 1 : (tiles + sms - 1) / sms;
      const int64_t t =
          waves * ((nkb + split - 1) / split * kb_cycles[i] + 2000) + (split > 1 ? 1500 : 0);
      if (t < best_t) {
        best_t = t;
        best = {widths[i], split};
      }
    }
  }
  return best;
}

template <bool QV>
cudaError_t launch_width(int bn, Fp8Args& a, const Operand& P, const Operand& Q, cudaStream_t s) {
  if constexpr (QV) {
    if (bn == 16) return launch_gemm<16, QV>(a, P, Q, s);
    if (bn == 32) return launch_gemm<32, QV>(a, P, Q, s);
  }
  if (bn == 64) return launch_gemm<64, QV>(a, P, Q, s);
  if (bn == 128) return launch_gemm<128, QV>(a, P, Q, s);
  return launch_gemm<256, QV>(a, P, Q, s);
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
  const int64_t kb = (K + BK - 1) / BK;
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
  const int es = c_dtype == MOE_DT_FP32 ? 4 : 2;
  if (!at(c, es) || !at(err, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  const Operand A = {a, M, lda, sa, ld_sa, true}, B = {b, N, ldb, sb, ld_sb, b_scale == 0};
  const bool swapped = M <= BM;
  const Operand &P = swapped ? B : A, &Q = swapped ? A : B;
  Fp8Args p = {};
  p.sp = P.s;
  p.sq = Q.s;
  p.ld_sp = P.ld_s;
  p.ld_sq = Q.ld_s;
  p.sp_vec = P.vec ? 1 : 0;
  p.swapped = swapped ? 1 : 0;
  p.c = c;
  p.ldc = ldc;
  p.c_fp32 = es == 4;
  p.align = at(c, 32) && ldc * es % 32 == 0 ? 32 : at(c, 16) && ldc * es % 16 == 0 ? 16 : 0;
  p.rows_p = (int)P.rows;
  p.rows_q = (int)Q.rows;
  p.K = (int)K;
  p.err = err;
  const Plan plan = choose(P.rows, Q.rows, kb, swapped && Q.vec, std::max(device_sms(), 1));
  p.tiles_p = (int)((P.rows + BM - 1) / BM);
  const int64_t tiles_q = (Q.rows + plan.bn - 1) / plan.bn;
  if (tiles_q * p.tiles_p > most) return fail(MOE_ERR_UNSUPPORTED, "too many tiles");
  p.tiles_q = (int)tiles_q;
  p.split = plan.split;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = Q.vec ? launch_width<true>(plan.bn, p, P, Q, s)
                        : launch_width<false>(plan.bn, p, P, Q, s);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 gemm launch");
  return MOE_OK;
}
