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
// kind::f8f6f4), warps 4-11 hold the 128 x BN fp32 sums (warp w: TMEM lanes 32 (w % 4).., half of
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
constexpr int kLeadWarps = 4;        // a warpgroup of its own: load, MMA, two idle
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;

struct Fp8Args {
  CUtensorMap tmP, tmQ;    // codes [rows, K]
  CUtensorMap tmSP, tmSQ;  // 1 x 128 scales [k-blocks, rows] (those that are vectors)
  const float* sp;         // 128 x 128 scales of P, [ceil(rows/128), k-blocks] (sp_vec = 0)
  const float* sq;         // 128 x 128 scales of Q (QV = 0)
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
  // Scale rows in flight. They are counted on the stage's barrier and have none of their own:
  // a stage is refilled for k-block n once the MMAs of n - STAGES are done, which were issued
  // after every epilogue warp had freed the buffer of n - STAGES - BUFS, hence was done with the
  // scales of the k-block before that.
  static constexpr int SLOTS = STAGES + BUFS + 1;
  static constexpr int SP_BYTES = BM * 4;
  static constexpr int SQ_BYTES = BN * 4 < 128 ? 128 : BN * 4;
  static constexpr int SLOT = SP_BYTES + SQ_BYTES;
  // Epilogue warps, and the registers of a thread: launched with 168 (384 threads of them fit an
  // SM), the lead warpgroup keeps 56 and each of the two epilogue warpgroups takes 224, for 128
  // sums and two TMEM loads of 32 columns in flight. Sixteen warps of 64 columns measured 5%
  // slower (8192 x 4096 x 14336: 343 us against 325), single loads of 64 columns the same (327).
  static constexpr int EW = 8;
  static constexpr int THREADS = 32 * (kLeadWarps + EW);
  static constexpr int LAUNCH_REGS = 65536 / THREADS / 8 * 8;
  static constexpr int LEAD_REGS = 56, EPI_REGS = 224;
  static_assert(32 * (kLeadWarps * LEAD_REGS + EW * EPI_REGS) <= THREADS * LAUNCH_REGS,
                "register split");
  static constexpr int GROUPS = EW / 4;                // column groups of a tile
  static constexpr int CW = BN / GROUPS;               // columns a warp holds
  static constexpr int SLOT_OFF = STAGES * STAGE;
  static constexpr int CTRL_OFF = SLOT_OFF + SLOTS * SLOT;
  static constexpr int TOTAL = CTRL_OFF + 512 + 1024;
  static_assert(TOTAL <= 232448, "shared memory above the per-block limit");
  static_assert(STAGES <= kMaxStages, "control block");
  static_assert(STAGES * STAGE >= BM * BN * 4, "the split sums fit in the stages");
};

struct Ctrl {
  uint64_t full[kMaxStages], empty[kMaxStages];
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

// True in one lane of a converged warp, the same one every time.
MOE_DEVICE bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Waits for this thread's TMEM loads; naming the registers keeps their uses behind the wait.
template <int W>
MOE_DEVICE void tmem_wait(uint32_t (&r)[W]) {
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < W; ++i) asm volatile("" : "+r"(r[i]));
}

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

// W consecutive results of one row.
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

// First row of P and of Q of a tile. Tiles are dealt in bands of kBand P tiles, Q tile by Q tile,
// so that the tiles in flight together read about as many rows of one side as of the other.
constexpr int kBand = 16;
template <int BN>
MOE_DEVICE void tile_at(const Fp8Args& p, int tile, int& p0, int& q0) {
  const int per = kBand * p.tiles_q, band = tile / per, in = tile - band * per;
  const int rows = min(kBand, p.tiles_p - band * kBand);
  p0 = (band * kBand + in % rows) * BM;
  q0 = (in / rows) * BN;
}

template <int BN, bool QV>
__global__ void __launch_bounds__(Smem<BN>::THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ Fp8Args p) {
  using L = Smem<BN>;
  constexpr int STAGES = L::STAGES, BUFS = L::BUFS, SLOTS = L::SLOTS;
  constexpr int CW = L::CW, CH = CW < 32 ? CW : 32;  // columns a warp holds, a TMEM load takes
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
    for (int s = 0; s < BUFS; ++s) {
      mbar_init(&c.tfull[s], 2);  // the MMAs, and the thread that saw the stage's scales land
      mbar_init(&c.tempty[s], L::EW);
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
  MOE_GRIDDEP_ENTRY();  // the setup above touches no global memory

  if (warp < kLeadWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(L::LEAD_REGS));
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      if (lane == 0) {
        const uint32_t tx = L::STAGE + (p.sp_vec ? L::SP_BYTES : 0) + (QV ? BN * 4 : 0);
        int stage = 0, slot = 0;
        uint32_t phase = 0;
        int64_t loaded = 0;  // k-blocks
        bool ok = true;
        for (int tile = tile0; ok && tile < total; tile += tstep) {
          int p0, q0;
          tile_at<BN>(p, tile, p0, q0);
          for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait(&c.empty[stage], phase ^ 1, abort, p.err)) {
              ok = false;
              break;
            }
            uint8_t* sP = smem + stage * L::STAGE;
            uint8_t* sl = smem + L::SLOT_OFF + slot * L::SLOT;
            uint64_t* bar = &c.full[stage];
            mbar_arrive_expect_tx(bar, tx);
            ++loaded;
            tma_load_2d(sP, &p.tmP, bar, kb * BK, p0);
            tma_load_2d(sP + L::P_BYTES, &p.tmQ, bar, kb * BK, q0);
            if (p.sp_vec) tma_load_2d(sl, &p.tmSP, bar, p0, kb);
            if (QV) tma_load_2d(sl + L::SP_BYTES, &p.tmSQ, bar, q0, kb);
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1;
            }
            if (++slot == SLOTS) slot = 0;
          }
        }
        // every load this thread issued lands before the CTA can exit: the last phase armed on
        // each barrier (load i of the ring sits at i % STAGES with parity (i / STAGES) & 1)
        const uint64_t t0 = globaltimer_ns();
        for (int64_t i = loaded > STAGES ? loaded - STAGES : 0; i < loaded; ++i)
          while (!mbar_try_wait(smem_u32(&c.full[i % STAGES]), (uint32_t)((i / STAGES) & 1)) &&
                 globaltimer_ns() - t0 < kWaitLimitNs) {
          }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // The warp stays together and one elected lane issues: addresses and descriptors are then
      // the same in every lane, which the MMAs' uniform operands need.
      const uint32_t tmem_u = __shfl_sync(0xFFFFFFFFu, tmem_base, 0);
      const uint64_t desc_p = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const int kb_short = p.K % BK ? nkb_all - 1 : -1;
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true, issued = false;
      for (int tile = tile0; ok && tile < total; tile += tstep) {
        for (int kb = kb0; kb < kb1; ++kb) {
          const bool got = mbar_wait(&c.tempty[buf], tphase ^ 1, abort, p.err) &&
                           mbar_wait(&c.full[stage], phase, abort, p.err);
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t dp = desc_p + (uint32_t)(stage * (L::STAGE >> 4));
          const uint64_t dq = dp + (L::P_BYTES >> 4);
          const uint32_t d = tmem_u + buf * BN;
          if (elect_one()) {
            if (kb != kb_short) {
#pragma unroll
              for (int ks = 0; ks < BK / MMA_K; ++ks)
                mma_f8_ss(d, dp + ks * (MMA_K >> 4), dq + ks * (MMA_K >> 4), idesc_f8(BM, BN),
                          ks != 0);
            } else {
              const int nsub = (p.K - kb * BK + MMA_K - 1) / MMA_K;
#pragma unroll 1
              for (int ks = 0; ks < nsub; ++ks)
                mma_f8_ss(d, dp + ks * (MMA_K >> 4), dq + ks * (MMA_K >> 4), idesc_f8(BM, BN),
                          ks != 0);
            }
            mma_commit(&c.empty[stage]);
            mma_commit(&c.tfull[buf]);
            mbar_arrive(&c.tfull[buf]);
          }
          __syncwarp();
          issued = true;
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
        if (elect_one()) mma_commit(&c.drain);
        __syncwarp();
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(smem_u32(&c.drain), 0) && globaltimer_ns() - t0 < kWaitLimitNs) {
        }
      }
      __syncwarp();
    }
    if (p.split > 1) {  // the epilogue warps' two cluster barriers
      cluster_sync_all();
      cluster_sync_all();
    }
  } else {
    // ------------------------------------------------------------ epilogue warps
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(L::EPI_REGS));
    const int q = warp & 3, c0 = ((warp - kLeadWarps) >> 2) * CW;  // lanes, first column
    const int row = q * 32 + lane;  // of the tile's P side
    constexpr int NC = CW / CH;     // TMEM loads a k-block
    const uint32_t tacc = tmem_base + c0 + ((uint32_t)(q * 32) << 16);
    int buf = 0, slot = 0;
    uint32_t tphase = 0;
    uint32_t r[2][CH];
    auto free_buffer = [&]() {  // its sums and scales have been read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.tempty[buf]);
      if (++buf == BUFS) {
        buf = 0;
        tphase ^= 1;
      }
    };
    // Waits for the next k-block and starts its first load. A wait that gives up has raised the
    // abort flag and the error word; the warps go on through their loops with undefined sums
    // (every later wait then returns at once), so no branch depends on it.
    auto next_block = [&]() {
      mbar_wait(&c.tfull[buf], tphase, abort, p.err);
      __syncwarp();
      tc_fence_after();
      tmem_ld(tacc + buf * BN, r[0]);
    };
    for (int tile = tile0; tile < total; tile += tstep) {
      __syncwarp();  // rows past the end left the last tile early
      int p0, q0;
      tile_at<BN>(p, tile, p0, q0);
      // Scales that are one number a k-block for these rows and columns (P's blocks when it has
      // no vector, times Q's): lane l holds that of k-block base + l. A column group past the
      // last column reads the last block's and stores nothing.
      const float* sp_at = p.sp_vec ? nullptr : p.sp + (int64_t)(p0 >> 7) * p.ld_sp;
      const float* sq_at =
          QV ? nullptr : p.sq + (int64_t)(min(q0 + c0, p.rows_q - 1) >> 7) * p.ld_sq;
      auto block_scales = [&](int base) {
        const int kb = min(base + lane, kb1 - 1);
        return (sp_at ? __ldg(sp_at + kb) : 1.0f) * (sq_at ? __ldg(sq_at + kb) : 1.0f);
      };
      float bs = block_scales(kb0);
      float acc[CW];
#pragma unroll
      for (int i = 0; i < CW; ++i) acc[i] = 0.f;
      next_block();
      for (int kb = kb0; kb < kb1; ++kb) {
        const int at = (kb - kb0) & 31;
        if (at == 0 && kb > kb0) bs = block_scales(kb);
        float f = __shfl_sync(0xFFFFFFFFu, bs, at);
        const float* sl = reinterpret_cast<const float*>(smem + L::SLOT_OFF + slot * L::SLOT);
        if (p.sp_vec) f *= sl[row];
        const float* sqv = sl + L::SP_BYTES / 4 + c0;
        if (++slot == SLOTS) slot = 0;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          tmem_wait(r[j & 1]);
          if (j + 1 < NC) {
            tmem_ld(tacc + buf * BN + (j + 1) * CH, r[(j + 1) & 1]);
          } else {
            free_buffer();
            // the next k-block's first load, before this one's last columns are added (an odd
            // number of loads a k-block would put it into the registers being added)
            if (NC % 2 == 0 && kb + 1 < kb1) next_block();
          }
#pragma unroll
          for (int i = 0; i < CH; i += 4) {
            float2 g0 = make_float2(f, f), g1 = g0;
            if (QV) {
              const float4 s4 = *reinterpret_cast<const float4*>(sqv + j * CH + i);
              g0 = __fmul2_rn(g0, make_float2(s4.x, s4.y));
              g1 = __fmul2_rn(g1, make_float2(s4.z, s4.w));
            }
            float* o = &acc[j * CH + i];
            const uint32_t* x = &r[j & 1][i];
            const float2 a0 = __ffma2_rn(make_float2(__uint_as_float(x[0]), __uint_as_float(x[1])),
                                         g0, make_float2(o[0], o[1]));
            const float2 a1 = __ffma2_rn(make_float2(__uint_as_float(x[2]), __uint_as_float(x[3])),
                                         g1, make_float2(o[2], o[3]));
            o[0] = a0.x;
            o[1] = a0.y;
            o[2] = a1.x;
            o[3] = a1.y;
          }
          if (NC % 2 == 1 && j + 1 == NC && kb + 1 < kb1) next_block();
        }
      }
      if (p.split > 1) {
        // this CTA's sums, column by column, where the stages were (every load has been used)
        float* st = reinterpret_cast<float*>(smem) + c0 * BM + row;
#pragma unroll
        for (int i = 0; i < CW; ++i) st[i * BM] = acc[i];
        break;  // one tile a cluster
      }
      if (p0 + row >= p.rows_p) continue;
      if (p.swapped) {
#pragma unroll
        for (int i = 0; i < CW; ++i) {
          const int64_t qr = q0 + c0 + i;
          if (qr < p.rows_q)
            store_swapped(p, p0 + row, qr, acc[i]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < CW / CH; ++j) {
          const int col = q0 + c0 + j * CH;
          if (col >= p.rows_q) break;
          float v[CH];
#pragma unroll
          for (int i = 0; i < CH; ++i) v[i] = acc[j * CH + i];
          store_row<CH>(p, p0 + row, col, v);
        }
      }
    }
    if (p.split > 1) {
      // rank r adds columns [r BN / split, (r + 1) BN / split) of every CTA of the cluster, in the
      // order of the ranks, and stores them
      __syncwarp();
      cluster_sync_all();
      if (!*abort) {
        const int tid = threadIdx.x - 32 * kLeadWarps;
        const int row = tid & 127, cg = tid >> 7;  // this thread's row, half of the columns
        int p0, q0;
        tile_at<BN>(p, tile0, p0, q0);
        const int per = BN / p.split;
        const uint32_t base = smem_u32(smem) + (uint32_t)row * 4;
        uint32_t peer[kMaxSplit];
#pragma unroll
        for (int s = 0; s < kMaxSplit; ++s)
          if (s < p.split) peer[s] = mapa_shared(base, (uint32_t)s);
        auto sum = [&](int col) {
          float v = 0.f;
#pragma unroll
          for (int s = 0; s < kMaxSplit; ++s)
            if (s < p.split) v += ld_shared_cluster(peer[s] + (uint32_t)col * (BM * 4));
          return v;
        };
        if (p0 + row < p.rows_p) {
          if (p.swapped) {
            const int half = per / 2;
            for (int i = rank * per + cg * half; i < rank * per + (cg + 1) * half; ++i)
              if (q0 + i < p.rows_q) store_swapped(p, p0 + row, q0 + i, sum(i));
          } else {  // 16 columns of a row at a time (per >= 16)
            for (int i = rank * per + cg * 16; i < (rank + 1) * per && q0 + i < p.rows_q; i += 32) {
              float v[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = sum(i + j);
              store_row<16>(p, p0 + row, q0 + i, v);
            }
          }
        }
        __syncwarp();
      }
      // no CTA leaves while another may read its sums
      cluster_sync_all();
    }
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
  // the register split waits for registers that the launch must have: checked once
  static const int regs = [&] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, kern) == cudaSuccess ? at.numRegs : 0;
  }();
  if (regs < Smem<BN>::LAUNCH_REGS) return cudaErrorInvalidConfiguration;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Smem<BN>::TOTAL);
  if (e != cudaSuccess) return e;
  const int tiles = a.tiles_p * a.tiles_q;
  const int sms = std::max(device_sms(), 1);
  const int grid = a.split > 1 ? tiles * a.split : std::min(tiles, sms);
  e = launch_pdl(kern, dim3((unsigned)grid), dim3(Smem<BN>::THREADS), Smem<BN>::TOTAL, s, a.split,
                 a);
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
      if (split > 1 && (tiles * split > sms || split > nkb || (!swapped && widths[i] / split < 16)))
        break;
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
