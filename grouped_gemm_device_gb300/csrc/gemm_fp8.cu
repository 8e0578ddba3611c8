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
//   Few rows (up to 64): P = b, Q = a (BN = M rounded up), so that the whole 128-row side is
//   filled with features and the small operand costs what it holds; the result is written
//   transposed, one feature a lane.
//   Tiles that do not fill the GPU (all of them, or those of the last round): the k-blocks are
//   split over a cluster of 2-8 CTAs, whose sums are added through distributed shared memory in
//   the order of their ranks.
//
// What bounds it. Many rows: a k-block of 128 x 256 moves 48 KB into shared memory and 48 KB out of
// it into the tensor cores, and its product waits for the sums of the one before the last to leave
// TMEM: 400 to 450 ns where the MMAs alone take about 300. 8192 x 14336 x 4096 (M x N x K): 345 to
// 380 us by what the power cap leaves, 2.5 to 2.8 PFLOP/s; 8192 x 4096 x 14336: 334 to 360 us, 2.7 to
// 2.9; 4096 x 4096 x 7168: 91 us, 2.6. Two 1 x 128 operands (weight gradients) need a second packed
// product a pair of results, and every lane reads every column's scale: 14336 x 4096 x 8192: 476 us,
// 2.0 PFLOP/s. Few rows: the weights' bytes and some 4 us of launch, first loads and cluster sums:
// with the weights from HBM (from L2) 1 x 4096 x 7168 9.1 us (7.6), 1 x 14336 x 4096 12.7 us (11.0),
// 4.6 TB/s (5.3), 128 x 4096 x 7168 12.3 us (10.9).
#include "gemm_common.cuh"
#include "realign.cuh"

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
  CUtensorMap tmSP, tmSQ;  // 1 x 128 scales [k-blocks, rows] (PV, QV)
  const float* sp;         // 128 x 128 scales of P, [ceil(rows/128), k-blocks] (not PV)
  const float* sq;         // the same of Q (not QV)
  int64_t ld_sp, ld_sq;
  int swapped;             // P = b, Q = a: C[q][p]
  void* c;
  int64_t ldc;
  int c_fp32;
  int align;               // bytes every row of C is aligned to (8, 16 or 32), or less
  int rows_p, rows_q, K;
  int tiles_p, tiles_q;
  // Every CTA takes `rounds` whole tiles; the `rem` tiles left go to one CTA each or, with
  // split > 1, to one cluster of that many CTAs each, which share the tile's k-blocks.
  int rounds, rem, split;
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

MOE_DEVICE void st_shared_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// W consecutive results of one row.
template <int W>
MOE_DEVICE void store_row(const Fp8Args& p, int64_t row, int col, const float (&v)[W]) {
  if (p.c_fp32) {
    float* o = static_cast<float*>(p.c) + row * p.ldc + col;
    if (p.align >= 16 && col + W <= p.rows_q) {
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
    if (p.align >= 16 && col + W <= p.rows_q) {
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
// n results of a row (at most W, fewer at the last column) as bf16, its address `o` on no 16-byte
// boundary: whole aligned blocks of 16 bytes, and element by element what is left at either end
// (4096 x 4092 x 4096: 184 us with every element by itself, 57 us for 4096 columns).
template <int W>
MOE_DEVICE void store_row_any(uint16_t* o, int n, const float (&v)[W]) {
  const int lead = lead_bytes(o);
  uint32_t last[4] = {0u, 0u, 0u, 0u};  // the eight results before
#pragma unroll
  for (int j = 0; j <= W; j += 8) {
    uint32_t w[8] = {last[0], last[1], last[2], last[3], 0u, 0u, 0u, 0u};
    if (j < W) {
#pragma unroll
      for (int i = 0; i < 4; ++i) last[i] = w[4 + i] = pack_bf16x2(v[j + 2 * i], v[j + 2 * i + 1]);
    }
    keep_bytes(w, lead);
    const int at = j - lead / 2;  // the block's first element
    if (at >= 0 && at + 8 <= n) {
      *reinterpret_cast<uint4*>(o + at) = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (at + i >= 0 && at + i < n) o[at + i] = (uint16_t)(w[4 + i / 2] >> (16 * (i & 1)));
    }
  }
}
// One result of the swapped form: row `prow` of P, row `qrow` of Q.
MOE_DEVICE void store_swapped(const Fp8Args& p, int prow, int64_t qrow, float v) {
  if (p.c_fp32) static_cast<float*>(p.c)[qrow * p.ldc + prow] = v;
  else static_cast<__nv_bfloat16*>(p.c)[qrow * p.ldc + prow] = __float2bfloat16_rn(v);
}

// First row of P and of Q of a tile. Tiles are dealt in bands of kBand P tiles, Q tile by Q tile,
// so that the tiles in flight together read about as many rows of one side as of the other (8192 x
// 14336 x 4096: 350 us, in bands of one 358).
constexpr int kBand = 16;
template <int BN>
MOE_DEVICE void tile_at(const Fp8Args& p, int tile, int& p0, int& q0) {
  const int per = kBand * p.tiles_q, band = tile / per, in = tile - band * per;
  const int rows = min(kBand, p.tiles_p - band * kBand);
  p0 = (band * kBand + in % rows) * BM;
  q0 = (in / rows) * BN;
}

// Four consecutive rows of P of the swapped form.
MOE_DEVICE void store_swapped4(const Fp8Args& p, int prow, int64_t qrow, float4 v) {
  const float x[4] = {v.x, v.y, v.z, v.w};
  if (p.align >= (p.c_fp32 ? 16 : 8) && prow + 4 <= p.rows_p) {
    if (p.c_fp32)
      *reinterpret_cast<float4*>(static_cast<float*>(p.c) + qrow * p.ldc + prow) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.c) + qrow * p.ldc + prow) =
          make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (prow + i < p.rows_p) store_swapped(p, prow + i, qrow, x[i]);
  }
}

// PV, QV: P and Q have 1 x 128 scales; otherwise 128 x 128.
template <int BN, bool PV, bool QV>
__global__ void __launch_bounds__(Smem<BN>::THREADS, 1)
    fp8_gemm_kernel(const __grid_constant__ Fp8Args p) {
  using L = Smem<BN>;
  constexpr int STAGES = L::STAGES, BUFS = L::BUFS, SLOTS = L::SLOTS;
  // columns a warp holds, and a TMEM load takes (with Q's scales beside them, half as many)
  constexpr int CW = L::CW, CH = CW < (QV ? 16 : 32) ? CW : (QV ? 16 : 32);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  Ctrl& c = *reinterpret_cast<Ctrl*>(smem + L::CTRL_OFF);
  volatile int* abort = &c.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nkb = (p.K + BK - 1) / BK;
  const int cluster = (int)blockIdx.x / p.split;
  const bool tail_split = p.split > 1 && cluster < p.rem;  // the same in a whole cluster
  // The it-th piece of work of this CTA: a tile and its k-blocks [k0, k1).
  auto unit = [&](int it, int& tile, int& k0, int& k1) {
    k0 = 0;
    k1 = nkb;
    tile = it * (int)gridDim.x + (int)blockIdx.x;
    if (it < p.rounds) return true;
    if (it > p.rounds) return false;
    if (p.split == 1) return (int)blockIdx.x < p.rem;
    const int rank = (int)blockIdx.x - cluster * p.split;
    tile = it * (int)gridDim.x + cluster;
    k0 = (int)((int64_t)nkb * rank / p.split);
    k1 = (int)((int64_t)nkb * (rank + 1) / p.split);
    return tail_split;
  };

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
        constexpr uint32_t tx = L::STAGE + (PV ? L::SP_BYTES : 0) + (QV ? BN * 4 : 0);
        int stage = 0, slot = 0;
        uint32_t phase = 0;
        int64_t loaded = 0;  // k-blocks
        bool ok = true;
        int tile, kb0, kb1;
        for (int it = 0; ok && unit(it, tile, kb0, kb1); ++it) {
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
            if (PV) tma_load_2d(sl, &p.tmSP, bar, p0, kb);
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
      const int kb_short = p.K % BK ? nkb - 1 : -1;
      int stage = 0, buf = 0;
      uint32_t phase = 0, tphase = 0;
      bool ok = true, issued = false;
      int tile, kb0, kb1;
      for (int it = 0; ok && unit(it, tile, kb0, kb1); ++it) {
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
    if (tail_split) {  // the epilogue warps' two cluster barriers
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
    constexpr bool kBlocks = !PV || !QV;  // one side has a number a k-block
    const float* const slots = reinterpret_cast<const float*>(smem + L::SLOT_OFF);
    const float* sl = slots;  // the next k-block's slot
    int buf = 0;
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
    // Starts on the next k-block of this warp's order: waits until its product is in `buf`,
    // starts the first load and fetches this row's scale. A wait that gives up has raised the
    // abort flag and the error word; the warps go on through their loops with undefined sums
    // (every later wait then returns at once), so no branch depends on it.
    auto start_block = [&](float& f, const float*& sqv) {
      mbar_wait(&c.tfull[buf], tphase, abort, p.err);
      __syncwarp();
      tc_fence_after();
      tmem_ld(tacc + buf * BN, r[0]);
      f = PV ? sl[row] : 1.0f;
      sqv = sl + L::SP_BYTES / 4 + c0;
      sl += L::SLOT / 4;
      if (sl == slots + SLOTS * (L::SLOT / 4)) sl = slots;
    };
    int tile, kb0, kb1;
    for (int it = 0; unit(it, tile, kb0, kb1); ++it) {
      __syncwarp();  // rows past the end left the last tile early
      int p0, q0;
      tile_at<BN>(p, tile, p0, q0);
      // Scales that are one number a k-block for these rows and columns (P's blocks when it has
      // no vector, times Q's): lane l holds that of k-block base + l. A column group past the
      // last column reads the last block's and stores nothing.
      const float* sp_at = PV ? nullptr : p.sp + (int64_t)(p0 >> 7) * p.ld_sp;
      const float* sq_at =
          QV ? nullptr : p.sq + (int64_t)(min(q0 + c0, p.rows_q - 1) >> 7) * p.ld_sq;
      auto block_scales = [&](int base) {
        const int kb = min(base + lane, kb1 - 1);
        return (PV ? 1.0f : __ldg(sp_at + kb)) * (QV ? 1.0f : __ldg(sq_at + kb));
      };
      float bs = kBlocks ? block_scales(kb0) : 1.0f, bs_next = 1.0f, f_next;
      const float* sq_next;
      float acc[CW];
#pragma unroll
      for (int i = 0; i < CW; ++i) acc[i] = 0.f;
      start_block(f_next, sq_next);
      for (int kb = kb0; kb < kb1; ++kb) {
        float f = f_next;
        const float* sqv = sq_next;
        const bool more = kb + 1 < kb1;
        const int at = (kb - kb0) & 31;
        float fb = 1.0f;
        if constexpr (kBlocks) {
          if (at == 0 && kb + 32 < kb1) bs_next = block_scales(kb + 32);  // one batch ahead
          fb = __shfl_sync(0xFFFFFFFFu, bs, at);
          if (at == 31) bs = bs_next;
        }
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          float4 s4[QV ? CH / 4 : 1];
          if constexpr (QV) {
#pragma unroll
            for (int i = 0; i < CH / 4; ++i)
              s4[i] = reinterpret_cast<const float4*>(sqv + j * CH)[i];
          }
          tmem_wait(r[j & 1]);
          if (j == 0) {
            // the scale's load is waited for here, not where it was issued
            asm volatile("" : "+f"(f));
            f *= fb;
          }
          if (j + 1 < NC) {
            tmem_ld(tacc + buf * BN + (j + 1) * CH, r[(j + 1) & 1]);
          } else {
            free_buffer();
            // the next k-block's first load, before this one's last columns are added (an odd
            // number of loads a k-block would put it into the registers being added)
            if (NC % 2 == 0 && more) start_block(f_next, sq_next);
          }
#pragma unroll
          for (int i = 0; i < CH; i += 4) {
            float2 g0 = make_float2(f, f), g1 = g0;
            if constexpr (QV) {
              g0 = __fmul2_rn(g0, make_float2(s4[i / 4].x, s4[i / 4].y));
              g1 = __fmul2_rn(g1, make_float2(s4[i / 4].z, s4[i / 4].w));
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
          if (NC % 2 == 1 && j + 1 == NC && more) start_block(f_next, sq_next);
        }
      }
      if (tail_split && it == p.rounds) {
        // Rank o adds up columns [o BN / split, (o + 1) BN / split): every CTA sends it its sums of
        // them (pushed: reading them from the other side measured 10 bytes a cycle), to
        // [rank][column][row] where the stages were, once every CTA is done with its stages.
        const int per = BN / p.split, lg = 31 - __clz(per);  // a power of two
        const uint32_t mine = smem_u32(smem) + (cluster_ctarank() * per * BM + row) * 4;
        constexpr int RUN = BN >= 64 ? 8 : 2;  // columns that surely have one owner
        __syncwarp();
        cluster_sync_all();
#pragma unroll
        for (int i = 0; i < CW; i += RUN) {
          const int owner = (c0 + i) >> lg;
          const uint32_t to =
              mapa_shared(mine + (uint32_t)(c0 + i - (owner << lg)) * (BM * 4), (uint32_t)owner);
#pragma unroll
          for (int j = 0; j < RUN; ++j) st_shared_cluster(to + j * (BM * 4), acc[i + j]);
        }
        break;  // the last of its work
      }
      if (p0 + row >= p.rows_p) continue;
      if (p.swapped) {
#pragma unroll
        for (int i = 0; i < CW; ++i) {
          const int64_t qr = q0 + c0 + i;
          if (qr < p.rows_q)
            store_swapped(p, p0 + row, qr, acc[i]);
        }
      } else if (p.align < 16 && !p.c_fp32) {
        const int col = q0 + c0, n = min(CW, p.rows_q - col);
        if (n > 0)
          store_row_any<CW>(
              static_cast<uint16_t*>(p.c) + (int64_t)(p0 + row) * p.ldc + col, n, acc);
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
    if (tail_split) {
      // the sums of this CTA's columns, in the order of the ranks
      __syncwarp();
      cluster_sync_all();
      if (!*abort) {
        const int w = warp - kLeadWarps, per = BN / p.split;
        const int col0 = (int)cluster_ctarank() * per;
        const float* sums = reinterpret_cast<const float*>(smem);
        int p0, q0;
        tile_at<BN>(p, tile, p0, q0);
        if (p.swapped) {  // four rows of P a lane
          const int prow = p0 + lane * 4;
          for (int i = w; i < per && q0 + col0 + i < p.rows_q; i += L::EW) {
            const float4* at = reinterpret_cast<const float4*>(sums + i * BM + lane * 4);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
            for (int s = 0; s < p.split; ++s, at += per * (BM / 4)) {
              const float4 x = *at;
              v.x += x.x;
              v.y += x.y;
              v.z += x.z;
              v.w += x.w;
            }
            if (prow < p.rows_p) store_swapped4(p, prow, q0 + col0 + i, v);
          }
        } else {  // eight columns of a row a lane (per is a multiple of 8)
          for (int u = w; u < 4 * (per / 8); u += L::EW) {
            const int r = (u & 3) * 32 + lane, i = (u >> 2) * 8;
            const float* x = sums + i * BM + r;
            float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int s = 0; s < p.split; ++s, x += per * BM)
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] += x[j * BM];
            if (p0 + r < p.rows_p && q0 + col0 + i < p.rows_q)
              store_row<8>(p, p0 + r, q0 + col0 + i, v);
          }
        }
        __syncwarp();
      }
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

// Clusters of `split` CTAs of a kernel that fit the GPU at once (1: CTAs).
template <int BN, bool PV, bool QV>
int resident(int split) {
  if (split == 1) return std::max(device_sms(), 1);
  static DeviceCache cache[kMaxSplit + 1];
  return std::max(1, cache[split].get(current_device(), [&] {
    auto kern = fp8_gemm_kernel<BN, PV, QV>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)split, 1, 1);
    cfg.blockDim = dim3(Smem<BN>::THREADS, 1, 1);
    cfg.dynamicSmemBytes = Smem<BN>::TOTAL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (ensure_smem_attr(reinterpret_cast<const void*>(kern), Smem<BN>::TOTAL) != cudaSuccess ||
        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
      cudaGetLastError();  // clear the sticky-free error of a failed query
      return 0;
    }
    return n;
  }));
}

struct Plan {
  int rounds = 0, rem = 0, split = 1, grid = 1;
  double ns = 1e30;
};

// How the tiles of one width are dealt out, by the time of the CTA that runs longest. A k-block of
// a 128 x BN tile was measured at `kb_ns`; a round's first loads and last stores at about 800 ns;
// adding up a cluster's sums at about 1200 ns and 11 ns a column of the tile.
template <int BN, bool PV, bool QV>
Plan plan_tiles(int64_t rows_p, int64_t rows_q, int64_t nkb) {
  constexpr double kb_ns = QV ? (BN >= 256 ? 620 : BN >= 128 ? 354 : BN >= 64 ? 300 : 265)
                              : (BN >= 256 ? 403 : BN >= 128 ? 286 : 262);
  const int64_t tiles = ((rows_p + BM - 1) / BM) * ((rows_q + BN - 1) / BN);
  Plan best;
  for (int split = 1; split <= kMaxSplit && split <= nkb; split *= 2) {
    const int64_t fit = resident<BN, PV, QV>(split), n = fit * split;
    Plan p;
    p.split = split;
    p.rounds = (int)(tiles / n);
    p.rem = (int)(tiles - p.rounds * n);
    if (split > 1 && (p.rem == 0 || p.rem > fit)) continue;
    p.grid = (int)(p.rounds ? n : (int64_t)p.rem * split);
    p.ns = p.rounds * (nkb * kb_ns + 800);
    if (p.rem) p.ns += (nkb + split - 1) / split * kb_ns + 800;
    if (split > 1) p.ns += 1200 + 11 * BN;
    if (p.ns < best.ns) best = p;
  }
  return best;
}

template <int BN, bool PV, bool QV>
cudaError_t launch_gemm(Fp8Args& a, const Plan& plan, const Operand& P, const Operand& Q,
                        cudaStream_t s) {
  const int64_t kb = (a.K + BK - 1) / BK;
  if (!tmap_codes(&a.tmP, P.q, P.rows, a.K, P.ld, BM) ||
      !tmap_codes(&a.tmQ, Q.q, Q.rows, a.K, Q.ld, BN) ||
      (PV && !tmap_scales(&a.tmSP, P.s, P.rows, kb, P.ld_s, BM)) ||
      (QV && !tmap_scales(&a.tmSQ, Q.s, Q.rows, kb, Q.ld_s, BN)))
    return cudaErrorInvalidValue;
  auto kern = fp8_gemm_kernel<BN, PV, QV>;
  // the register split waits for registers that the launch must have
  static DeviceCache cache;
  cudaError_t e = cudaSuccess;
  const int regs = cache.get(current_device(), [&] {
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, kern);
    return e == cudaSuccess ? at.numRegs : 0;
  });
  if (e != cudaSuccess) return e;
  if (regs < Smem<BN>::LAUNCH_REGS) return cudaErrorInvalidConfiguration;
  e = ensure_smem_attr(reinterpret_cast<const void*>(kern), Smem<BN>::TOTAL);
  if (e != cudaSuccess) return e;
  a.tiles_p = (int)((P.rows + BM - 1) / BM);
  a.tiles_q = (int)((Q.rows + BN - 1) / BN);
  a.rounds = plan.rounds;
  a.rem = plan.rem;
  a.split = plan.split;
  e = launch_pdl(kern, dim3((unsigned)plan.grid), dim3(Smem<BN>::THREADS), Smem<BN>::TOTAL, s,
                 a.split, a);
  count_launch(s, MOE_K_FP8_GEMM);
  return e;
}

// Whether the swapped form is taken: up to 32 rows always, up to 64 where the 128-feature tiles give
// every CTA pair of SMs at most one and K has 12 k-blocks. Its tiles stay a load long, while many
// of 64 rows write 64 transposed results a feature; with few k-blocks that is most of the time.
// Measured with operands from HBM, swapped and not, us (M x N x K):
//   32 x 4096 x 7168 9.7, 11.9    64 x 4096 x 7168 10.6, 12.1    64 x 14336 x 4096 15.4, 14.5
//   32 x 14336 x 4096 13.9, 13.9  64 x 8192 x 8192 16.3, 20.4    64 x 32768 x 4096 29.0, 26.0
//   32 x 1024 x 1024 4.3, 4.6     64 x 9728 x 4096 11.7, 12.5    64 x 9856 x 2048 9.7, 8.6
//   32 x 2048 x 512 4.2, 3.5      64 x 2048 x 1536 5.7, 6.0      64 x 4096 x 1152 7.4, 5.9
// (the rule loses at 32 x 2048 x 512, and 64 x 7168 x 2048: 8.1, 7.6).
bool few_rows(int64_t M, int64_t N, int64_t K) {
  return M <= 32 || (M <= 64 && (N + BM - 1) / BM * 2 <= device_sms() && K >= 12 * BK);
}

// The widths in turn: the one whose plan ends first. Few rows take the narrowest tile that holds
// them (swapped form); otherwise
// tiles of 64, 128 or 256 columns.
template <bool PV, bool QV>
cudaError_t launch_any(Fp8Args& a, const Operand& P, const Operand& Q, cudaStream_t s) {
  const int64_t nkb = (a.K + BK - 1) / BK;
  if (a.swapped) {
    if constexpr (QV) {
      if (Q.rows <= 16)
        return launch_gemm<16, PV, QV>(a, plan_tiles<16, PV, QV>(P.rows, Q.rows, nkb), P, Q, s);
      if (Q.rows <= 32)
        return launch_gemm<32, PV, QV>(a, plan_tiles<32, PV, QV>(P.rows, Q.rows, nkb), P, Q, s);
      return launch_gemm<64, PV, QV>(a, plan_tiles<64, PV, QV>(P.rows, Q.rows, nkb), P, Q, s);
    }
  } else if constexpr (PV) {
    const Plan p64 = plan_tiles<64, PV, QV>(P.rows, Q.rows, nkb);
    const Plan p128 = plan_tiles<128, PV, QV>(P.rows, Q.rows, nkb);
    const Plan p256 = plan_tiles<256, PV, QV>(P.rows, Q.rows, nkb);
    if (p256.ns <= p128.ns && p256.ns <= p64.ns)
      return launch_gemm<256, PV, QV>(a, p256, P, Q, s);
    if (p128.ns <= p64.ns) return launch_gemm<128, PV, QV>(a, p128, P, Q, s);
    return launch_gemm<64, PV, QV>(a, p64, P, Q, s);
  }
  return cudaErrorInvalidValue;  // a (Q when swapped, else P) always has 1 x 128 scales
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
  const bool swapped = few_rows(M, N, K);
  const Operand &P = swapped ? B : A, &Q = swapped ? A : B;
  if ((P.rows + BM - 1) / BM * ((Q.rows + 15) / 16) > most)
    return fail(MOE_ERR_UNSUPPORTED, "too many tiles");
  Fp8Args p = {};
  p.sp = P.s;
  p.sq = Q.s;
  p.ld_sp = P.ld_s;
  p.ld_sq = Q.ld_s;
  p.swapped = swapped ? 1 : 0;
  p.c = c;
  p.ldc = ldc;
  p.c_fp32 = es == 4;
  p.align = 32;
  while (p.align > es && (!at(c, p.align) || ldc * es % p.align)) p.align /= 2;
  p.rows_p = (int)P.rows;
  p.rows_q = (int)Q.rows;
  p.K = (int)K;
  p.err = err;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = !Q.vec  ? launch_any<true, false>(p, P, Q, s)
                  : P.vec ? launch_any<true, true>(p, P, Q, s)
                          : launch_any<false, true>(p, P, Q, s);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 gemm launch");
  return MOE_OK;
}
