// The residual stream around a block and its two root-mean-square norms, forward and backward
// (moe_residual_norm_fwd / moe_residual_norm_bwd in include/moegmm.h).
//
//   u = wp o rp,  x' = x + s g u,  h = w x' r;       rp, r = 1 / sqrt(mean(.^2) + eps)
//   y = x' r, z = o rp:  dx = dx' + r (dh w - y mean(dh w y));  e = dx wp
//   do = s g rp (e - z mean(e z));  dg = s sum(e z);  dwp = sum_m s g dx z;  dw = sum_m dh y
//
// Bound by HBM: the forward reads x and o and writes x' and h, the backward reads dh, dx', x' and
// o and writes dx and do. A row stays in registers (forward) or in shared memory (backward)
// between its sums and their use; statistics, sums and the weights' gradients are fp32. 16384 x
// 2880, fp32 stream and bf16 branches, both norms and a gate: forward 87 us, 6.5 TB/s, 97% of the
// measured copy; 8192 x 4095 bf16, both norms and a gate, forward 74 us, 3.6 TB/s (partial vectors).
// 8192 x 4096 bf16 backward 67 us, 6.0 TB/s, 5 of them the sum of the partial
// weight gradients; 3001 x 4095 bf16, both norms and a gate, backward 43 us, 3.5 TB/s: ten rows a
// block, two barriers a row and the handling of partial vectors. Backward with fewer rows ahead and
// one block an SM: 16384 x 2880 fp32 stream, bf16 branches, both norms and a gate 235 us (floor 127);
// 4096 x 7168 of those types 122 (79), in fp32 throughout 201 (105); 2048 x 16384 bf16 123 (60). One
// row of 7168: forward 5.3 us, backward 8.4, the host's.
#include "kernels.cuh"
#include "row8.cuh"

namespace moe {
namespace {

struct FwdArgs {
  const void *x, *o;
  void *xn, *h;
  int64_t ldx, ldo, ldxn, ldh, M, N;
  Weight wp, w;
  const float* gate;
  float *rstd_post, *rstd;
  float scale, eps;
  int post;
};

// Any length, stride and place: a block a row, element by element, the row once for each sum and
// once for each result (the later ones from L2). 8192 x 4095 bf16 with branches 4104 apart: forward
// 200 us, floor 40, and backward (rn_bwd_any_kernel) 501, floor 60; 2048 x 16384 fp32 backward 660,
// floor 120.
template <typename XT, typename OT>
__global__ void __launch_bounds__(1024) rn_fwd_any_kernel(const FwdArgs a) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[2][32];
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
    const OT* o = static_cast<const OT*>(a.o) + row * a.ldo;
    XT* xn = static_cast<XT*>(a.xn) + row * a.ldxn;
    float rp = 1.0f;
    if (a.post) {
      float s = 0.f;
      for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
        const float v = to_float(o[c]);
        s += v * v;
      }
      rp = 1.0f / sqrtf(group_sum<1024>(s, sm[0]) / (float)a.N + a.eps);
      if (threadIdx.x == 0 && a.rstd_post) a.rstd_post[row] = rp;
    }
    const float q = a.gate ? a.scale * a.gate[row] : a.scale;
    float s = 0.f;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
      XT v = x[c];
      if (a.o) {
        const float z = a.post ? to_float(o[c]) * rp : to_float(o[c]);
        v = from_float<XT>(to_float(v) + q * (z * weight_at(a.wp, c)));
        xn[c] = v;
      }
      s += to_float(v) * to_float(v);
    }
    if (a.h) {
      const float r = 1.0f / sqrtf(group_sum<1024>(s, sm[1]) / (float)a.N + a.eps);
      if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
      const XT* y = a.o ? xn : x;
      for (int64_t c = threadIdx.x; c < a.N; c += 1024)
        static_cast<OT*>(a.h)[row * a.ldh + c] = from_float<OT>(to_float(y[c]) * r * weight_at(a.w, c));
    }
    __syncthreads();  // the sums' places are used again
  }
}

// A row of up to 8 G PER columns (ANY: 7 less) in the registers of G threads, a warp of four in a
// block or a whole block: read once, both sums taken, written once.
template <typename XT, typename OT, int G, int PER, bool ANY>
__global__ void __launch_bounds__(G < 128 ? 128 : G) rn_fwd_kernel(const FwdArgs a) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[2][32];
  constexpr int R = G < 128 ? 128 / G : 1;
  const int t = threadIdx.x % G, N = (int)a.N;
  const int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / G;
  if (G == 32 && row >= a.M) return;  // a block's groups are its warps; otherwise R = 1
  const XT* x = static_cast<const XT*>(a.x) + row * a.ldx;
  const OT* o = static_cast<const OT*>(a.o) + row * a.ldo;
  const int lead = ANY ? lead8(x) : 0;
  Raw8<XT> xr[PER];
  Raw8<OT> br[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (i * G + t) * 8 - lead;
    zero8(xr[i]);
    zero8(br[i]);
    if (c < N) {
      if (a.o) load8(o + c, br[i]);
      load8(x + c, xr[i]);
      if (ANY && (c < 0 || c + 8 > N)) {
        clear8(br[i], -c, N - c);
        clear8(xr[i], -c, N - c);
      }
    }
  }
  float s = 0.f;
  if (a.o) {
    float rp = 1.0f;
    if (a.post) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s += at8(br[i], j) * at8(br[i], j);
      rp = 1.0f / sqrtf(group_sum<G>(s, sm[0]) / (float)N + a.eps);
      if (t == 0 && a.rstd_post) a.rstd_post[row] = rp;
    }
    const float q = (a.gate ? a.scale * a.gate[row] : a.scale) * rp;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * 8 - lead;
      if (c < N) {
        float wp[8], v[8];
        weights8<ANY>(a.wp, c, N, wp);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = at8(xr[i], j) + q * (at8(br[i], j) * wp[j]);
        round8(v, xr[i]);
        store8<ANY>(static_cast<XT*>(a.xn) + row * a.ldxn + c, xr[i], -c, N - c);
      }
    }
  }
  if (!a.h) return;
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s += at8(xr[i], j) * at8(xr[i], j);
  const float r = 1.0f / sqrtf(group_sum<G>(s, sm[1]) / (float)N + a.eps);
  if (t == 0 && a.rstd) a.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int c = (i * G + t) * 8 - lead;
    if (c < N) {
      float w[8];
      weights8<ANY>(a.w, c, N, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= at8(xr[i], j) * r;
      Raw8<OT> hr;
      round8(w, hr);
      store8<ANY>(static_cast<OT*>(a.h) + row * a.ldh + c, hr, -c, N - c);
    }
  }
}

// A row of partial sums: whole vectors, and the place of a row's first element in its first one.
template <typename I>
__host__ __device__ constexpr I part_pitch(I N) {
  return (N + 7) / 8 * 8 + 8;
}
// Eight partial sums. The workspace lies on any 16-byte boundary; on a 32-byte one they are a single
// store (8192 x 4096 bf16 backward 66.8 us, 68.0 with two everywhere).
MOE_DEVICE void store_part8(float* p, const float (&v)[8]) {
  if ((reinterpret_cast<uintptr_t>(p) & 31u) == 0) {
    Raw8<float> r;
    round8(v, r);
    store8<false>(p, r, 0, 8);
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
struct BwdArgs {
  const void *dh, *dxn, *xn, *o;
  void *dx, *d_o;
  int64_t lddh, lddxn, ldxn, ldo, lddx, lddo, M, N;
  Weight wp, w;
  const float *gate, *rstd_post, *rstd;
  float* d_gate;
  float scale;
  int post;
  float* part;  // [blocks][2][part_pitch(N)]: dw, dwp
  void *dw, *dwp;
  int w_fp32;
};

template <typename XT, typename OT>
__global__ void __launch_bounds__(1024) rn_bwd_any_kernel(const BwdArgs a) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[2][32];
  const int64_t NP = part_pitch(a.N);
  float* part = a.part ? a.part + (int64_t)blockIdx.x * 2 * NP : nullptr;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
    const OT* dh = static_cast<const OT*>(a.dh) + row * a.lddh;
    const XT* dxn = static_cast<const XT*>(a.dxn) + row * a.lddxn;
    const XT* xn = static_cast<const XT*>(a.xn) + row * a.ldxn;
    const OT* o = static_cast<const OT*>(a.o) + row * a.ldo;
    const float r = a.dh ? a.rstd[row] : 0.f, rp = a.post ? a.rstd_post[row] : 1.0f;
    const float q = a.gate ? a.scale * a.gate[row] : a.scale;
    float c1 = 0.f;
    if (a.dh) {
      for (int64_t c = threadIdx.x; c < a.N; c += 1024)
        c1 += to_float(dh[c]) * weight_at(a.w, c) * (to_float(xn[c]) * r);
      c1 = group_sum<1024>(c1, sm[0]) / (float)a.N;
    }
    auto grad = [&](int64_t c) {
      float d = a.dxn ? to_float(dxn[c]) : 0.f;
      if (a.dh) d += r * (to_float(dh[c]) * weight_at(a.w, c) - to_float(xn[c]) * r * c1);
      return d;
    };
    float dot = 0.f;
    if (a.o && (a.post || a.d_gate)) {
      for (int64_t c = threadIdx.x; c < a.N; c += 1024)
        dot += grad(c) * weight_at(a.wp, c) * (to_float(o[c]) * rp);
      dot = group_sum<1024>(dot, sm[1]);
      if (threadIdx.x == 0 && a.d_gate) a.d_gate[row] = a.scale * dot;
    }
    const float c2 = a.post ? dot / (float)a.N : 0.f;
    for (int64_t c = threadIdx.x; c < a.N; c += 1024) {
      const float d = grad(c);
      const float y = a.dh ? to_float(xn[c]) * r : 0.f, dw = a.dh ? to_float(dh[c]) * y : 0.f;
      const float z = a.o ? to_float(o[c]) * rp : 0.f, dwp = q * d * z;
      if (part) {  // column c belongs to this thread in every row
        part[c] = first ? dw : part[c] + dw;
        part[NP + c] = first ? dwp : part[NP + c] + dwp;
      }
      if (a.dx) static_cast<XT*>(a.dx)[row * a.lddx + c] = from_float<XT>(d);
      if (a.d_o)
        static_cast<OT*>(a.d_o)[row * a.lddo + c] =
            from_float<OT>(q * rp * (d * weight_at(a.wp, c) - z * c2));
    }
    first = false;
    __syncthreads();
  }
}


// Threads a block of the kernel that walks rows: eight warps with a row each, or one row.
constexpr int block_of(int G) { return G == 32 ? 256 : G; }
template <int N>
MOE_DEVICE void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
MOE_DEVICE void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16-byte units of a vector of the four tensors that are read: x_new, dx_new, o, dh.
template <typename XT, typename OT>
constexpr int units() {
  return (int)(sizeof(XT) + sizeof(OT));
}

// The weights of the elements that wrap: those of columns c .. N - 1 come first.
MOE_DEVICE void wrap_weights(const Weight& w, int N, int c, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < N) v[j] = weight_at(w, c + j);
}

// A group of G threads walks rows that lie alike in their vectors; a thread owns the same 8 PER
// columns of every row and keeps their sums of the weights' gradients in registers until the end.
// Each thread copies its own columns of the next S - 1 rows into a ring in shared memory
// (cp.async), so that no barrier is spent on the copies. Where a row's bytes leave room for one row
// alone (S = 1: bf16 branches above 8192 columns; fp32 ones of 257 to 512 and of 2049 to 8192) none is
// ahead, and a row is waited for as soon as it is asked for. N <= 8 G PER, and the groups' number a
// multiple of 8 where ANY and a group takes more than one row. ANY: a row may reach into one
// vector more than the group's; its elements there are fewer than those that the first vector's
// `lead` leaves free, and wrap around to them. Two blocks an SM (ANY, 256 threads): 3001 x 4095 42
// us against 54 with the registers it would take.
template <typename XT, typename OT, int G, int PER, int S, bool ANY>
__global__ void __launch_bounds__(block_of(G), ANY && G == 256 ? 2 : 1)
    rn_bwd_kernel(const BwdArgs a) {
  MOE_GRIDDEP_ENTRY();
  constexpr int B = block_of(G), GROUPS = B / G, U = units<XT, OT>();
  constexpr int UX = sizeof(XT) / 2, UO = sizeof(OT) / 2;
  // few enough columns a thread to hold both weights beside the sums
  constexpr bool kKeep = PER <= 2 && G <= 512;
  __shared__ float sm[2][2][32];
  extern __shared__ uint4 ring[];  // [S][PER][U][B]; ANY: [S][GROUPS][U] for the vectors that wrap
  constexpr int CAP = 8 * G * PER;
  uint4* spare = ring + S * PER * U * B + threadIdx.x / G * U;
  const int t = threadIdx.x % G, N = (int)a.N;
  const int64_t row0 = (int64_t)blockIdx.x * GROUPS + threadIdx.x / G;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const XT* xn = static_cast<const XT*>(a.xn);
  const XT* dxn = static_cast<const XT*>(a.dxn);
  const OT* o = static_cast<const OT*>(a.o);
  const OT* dh = static_cast<const OT*>(a.dh);
  const int lead = !ANY ? 0
                   : dh ? lead8(dh + row0 * a.lddh)
                        : lead8(dxn + row0 * a.lddxn);
  const bool wraps = ANY && t == 0 && CAP - lead < N;
  // the vector of columns c .. c + 7 to units `pitch` bytes apart
  auto copy = [&](int64_t row, int c, uint32_t at, uint32_t pitch) {
#pragma unroll
    for (int u = 0; u < UX; ++u) {
      if (dh) cp_async16(at + u * pitch, reinterpret_cast<const uint4*>(xn + row * a.ldxn + c) + u);
      if (dxn)
        cp_async16(at + (UX + u) * pitch,
                   reinterpret_cast<const uint4*>(dxn + row * a.lddxn + c) + u);
    }
#pragma unroll
    for (int u = 0; u < UO; ++u) {
      if (o)
        cp_async16(at + (2 * UX + u) * pitch,
                   reinterpret_cast<const uint4*>(o + row * a.ldo + c) + u);
      if (dh)
        cp_async16(at + (2 * UX + UO + u) * pitch,
                   reinterpret_cast<const uint4*>(dh + row * a.lddh + c) + u);
    }
  };
  auto fetch = [&](int64_t row, int slot) {
    if (row < a.M) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int c = (i * G + t) * 8 - lead;
        if (c < N)
          copy(row, c, smem_u32(ring) + (((slot * PER + i) * U) * B + threadIdx.x) * 16, B * 16);
      }
      if (wraps) copy(row, CAP - lead, smem_u32(spare + slot * GROUPS * U), 16);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // vector i of a row's tensor that begins at unit `first`; zeros where there is none
  auto take = [&](auto& r, bool there, int slot, int i, int first) {
    constexpr int W = sizeof(r.w) / 16;
    zero8(r);
    if (!there) return;
#pragma unroll
    for (int u = 0; u < W; ++u) {
      const uint4 q = ring[((slot * PER + i) * U + first + u) * B + threadIdx.x];
      r.w[4 * u] = q.x;
      r.w[4 * u + 1] = q.y;
      r.w[4 * u + 2] = q.z;
      r.w[4 * u + 3] = q.w;
    }
  };
  // What a row's first and last vector hold of other rows is cleared in the ring, once a row, and
  // what wraps put there.
  auto clear = [&](auto r, int slot, int i, int first, int c) {
    take(r, true, slot, i, first);
    clear8(r, -c, N - c);
    if (wraps && i == 0) {
      auto more = r;
#pragma unroll
      for (int u = 0; u < (int)sizeof(r.w) / 16; ++u) {
        const uint4 q = spare[slot * GROUPS * U + first + u];
        more.w[4 * u] = q.x;
        more.w[4 * u + 1] = q.y;
        more.w[4 * u + 2] = q.z;
        more.w[4 * u + 3] = q.w;
      }
      clear8(more, 0, N - (CAP - lead));  // fewer than lead are left
#pragma unroll
      for (int k = 0; k < (int)sizeof(r.w) / 4; ++k) r.w[k] |= more.w[k];
    }
#pragma unroll
    for (int u = 0; u < (int)sizeof(r.w) / 16; ++u)
      ring[((slot * PER + i) * U + first + u) * B + threadIdx.x] =
          make_uint4(r.w[4 * u], r.w[4 * u + 1], r.w[4 * u + 2], r.w[4 * u + 3]);
  };
  auto clear_edges = [&](int slot) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * 8 - lead;
      if (c >= N || (c >= 0 && c + 8 <= N)) continue;
      clear(Raw8<XT>(), slot, i, 0, c);
      clear(Raw8<XT>(), slot, i, UX, c);
      clear(Raw8<OT>(), slot, i, 2 * UX, c);
      clear(Raw8<OT>(), slot, i, 2 * UX + UO, c);
    }
  };
  float dw[PER][8], dwp[PER][8], w_[kKeep ? PER : 1][8], wp_[kKeep ? PER : 1][8];
#pragma unroll
  for (int i = 0; i < PER; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = dwp[i][j] = 0.f;
#pragma unroll
  for (int k = 0; k < S - 1; ++k) fetch(row0 + k * step, k);
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * 8 - lead;
      if (c < N) {
        weights8<ANY>(a.w, c, N, w_[i]);
        weights8<ANY>(a.wp, c, N, wp_[i]);
        if (wraps && i == 0) {
          wrap_weights(a.w, N, CAP - lead, w_[i]);
          wrap_weights(a.wp, N, CAP - lead, wp_[i]);
        }
      }
    }
  }
  auto weight = [&](const Weight& w, float (&kept)[kKeep ? PER : 1][8], int i, float (&v)[8]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = kept[i][j];
    } else {
      weights8<ANY>(w, (i * G + t) * 8 - lead, N, v);
      if (wraps && i == 0) wrap_weights(w, N, CAP - lead, v);
    }
  };
  int slot = 0, turn = 0;
  for (int64_t row = row0; row < a.M; row += step) {
    const float r = dh ? a.rstd[row] : 0.f, rp = a.post ? a.rstd_post[row] : 1.0f;
    const float q = a.gate ? a.scale * a.gate[row] : a.scale;
    fetch(row + (S - 1) * step, slot == 0 ? S - 1 : slot - 1);
    cp_async_wait<S - 1>();
    if (ANY) clear_edges(slot);
    float c1 = 0.f;
    if (dh) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if ((i * G + t) * 8 - lead >= N) continue;
        Raw8<XT> xr;
        Raw8<OT> hr;
        float w[8];
        take(xr, true, slot, i, 0);
        take(hr, true, slot, i, 2 * UX + UO);
        weight(a.w, w_, i, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float y = at8(xr, j) * r, g = at8(hr, j);
          dw[i][j] += g * y;
          c1 += (g * w[j]) * y;
        }
      }
      c1 = group_sum<G>(c1, sm[turn][0]) / (float)N;
    }
    float d[PER][8], dot = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int c = (i * G + t) * 8 - lead;
      if (c >= N) continue;
      Raw8<XT> xr, dr;
      Raw8<OT> hr, br;
      float w[8], wp[8];
      take(xr, dh != nullptr, slot, i, 0);
      take(dr, dxn != nullptr, slot, i, UX);
      take(br, o != nullptr, slot, i, 2 * UX);
      take(hr, dh != nullptr, slot, i, 2 * UX + UO);
      weight(a.w, w_, i, w);
      weight(a.wp, wp_, i, wp);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        d[i][j] = at8(dr, j) + r * (at8(hr, j) * w[j] - (at8(xr, j) * r) * c1);
        const float z = at8(br, j) * rp;
        dwp[i][j] += (q * d[i][j]) * z;
        dot += (d[i][j] * wp[j]) * z;
      }
      if (a.dx) {
        round8(d[i], dr);
        store8<ANY>(static_cast<XT*>(a.dx) + row * a.lddx + c, dr, -c, N - c);
        if (wraps && i == 0)
          store8<ANY>(static_cast<XT*>(a.dx) + row * a.lddx + CAP - lead, dr, 0, N - CAP + lead);
      }
    }
    if (o) {
      if (a.post || a.d_gate) {
        dot = group_sum<G>(dot, sm[turn][1]);
        if (t == 0 && a.d_gate) a.d_gate[row] = a.scale * dot;
      }
      if (a.d_o) {
        const float c2 = a.post ? dot / (float)N : 0.f, qr = q * rp;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const int c = (i * G + t) * 8 - lead;
          if (c >= N) continue;
          Raw8<OT> br;
          float wp[8];
          take(br, true, slot, i, 2 * UX);
          weight(a.wp, wp_, i, wp);
#pragma unroll
          for (int j = 0; j < 8; ++j) wp[j] = qr * (d[i][j] * wp[j] - (at8(br, j) * rp) * c2);
          round8(wp, br);
          store8<ANY>(static_cast<OT*>(a.d_o) + row * a.lddo + c, br, -c, N - c);
          if (wraps && i == 0)
            store8<ANY>(static_cast<OT*>(a.d_o) + row * a.lddo + CAP - lead, br, 0,
                        N - CAP + lead);
        }
      }
    }
    turn ^= 1;
    if (++slot == S) slot = 0;
  }
  cp_async_wait<0>();
  if (!a.part) return;
  // the column of element j of vector i, -1 past the row's ends
  auto column = [&](int i, int j) {
    int c = (i * G + t) * 8 - lead + j;
    if (ANY && c < 0) c += CAP;
    return c < N && (c >= 0) ? c : -1;
  };
  // a block's sums to its partials, or (a single block) the results
  float* part = a.part + (int64_t)blockIdx.x * 2 * part_pitch(N);
  auto put = [&](int c, float x, float y) {
    if (gridDim.x > 1) {
      part[c] = x;
      part[part_pitch(N) + c] = y;
    } else if (a.w_fp32) {
      if (a.dw) static_cast<float*>(a.dw)[c] = x;
      if (a.dwp) static_cast<float*>(a.dwp)[c] = y;
    } else {
      if (a.dw) static_cast<__nv_bfloat16*>(a.dw)[c] = __float2bfloat16_rn(x);
      if (a.dwp) static_cast<__nv_bfloat16*>(a.dwp)[c] = __float2bfloat16_rn(y);
    }
  };
  if constexpr (GROUPS > 1) {
    // the block's groups, in order, through the columns of one shared row at a time
    __shared__ float cols[2][G * PER * 8];
    for (int g = 0; g < GROUPS; ++g) {
      __syncthreads();
      if ((int)threadIdx.x / G == g) {
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = column(i, j);
            if (c < 0) continue;
            cols[0][c] = g == 0 ? dw[i][j] : cols[0][c] + dw[i][j];
            cols[1][c] = g == 0 ? dwp[i][j] : cols[1][c] + dwp[i][j];
          }
      }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < N; c += B) put(c, cols[0][c], cols[1][c]);
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int at = (i * G + t) * 8;
      if (at - lead >= N) continue;
      if (gridDim.x > 1) {  // column c at c + lead: whole vectors
        store_part8(part + at, dw[i]);
        store_part8(part + part_pitch(N) + at, dwp[i]);
        if (wraps && i == 0) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < lead && column(i, j) >= 0) put(CAP + j, dw[i][j], dwp[i][j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (column(i, j) >= 0) put(column(i, j), dw[i][j], dwp[i][j]);
      }
    }
  }
}

// dw (columns [0, N)) and dwp (columns [N, 2 N)) = sum of the blocks' partials in a fixed order;
// block b's column c lies at c + (place + b pitch) % 8. Each of a block's 32 warps sums every 32nd
// partial of 32 columns; the warps' sums are added as a tree.
template <typename WT>
__global__ void __launch_bounds__(1024) rn_colsum_kernel(const float* __restrict__ part,
                                                         int nparts, int64_t N,
                                                         WT* __restrict__ dw,
                                                         WT* __restrict__ dwp, uint32_t place,
                                                         uint32_t pitch) {
  MOE_GRIDDEP_ENTRY();
  __shared__ float sm[32][33];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int64_t c = (int64_t)blockIdx.x * 32 + lane, NP = part_pitch(N);
  float s = 0.f;
  if (c < 2 * N) {
    const float* at = part + (c < N ? c : c - N + NP);
#pragma unroll 5
    for (int b = w; b < nparts; b += 32)
      s += at[(int64_t)b * 2 * NP + ((place + (uint32_t)b * pitch) & 7u)];
  }
  sm[w][lane] = s;
  __syncthreads();
  s = sm[lane][w];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  const int64_t col = (int64_t)blockIdx.x * 32 + w;
  if (lane == 0 && col < 2 * N) {
    if (col < N) {
      if (dw) dw[col] = from_float<WT>(s);
    } else if (dwp) {
      dwp[col - N] = from_float<WT>(s);
    }
  }
}

constexpr int64_t kMaxParts = 480;  // rows of partial weight gradients

// Whether every row of a tensor lies in its vectors as those of the first one given do.
struct Places {
  bool first = true, same = true, aligned = true;
  int64_t place = 0, pitch = 0;
  void add(const void* p, int64_t ld, int bytes) {
    if (!p) return;
    const int64_t at = (int64_t)(reinterpret_cast<uintptr_t>(p) / bytes & 7u);
    if (first) {
      place = at;
      pitch = ld & 7;
      first = false;
    }
    same = same && at == place && (ld & 7) == pitch;
    aligned = aligned && at == 0 && (ld & 7) == 0;
  }
};

template <typename XT, typename OT, bool ANY, int G, int PER>
cudaError_t fwd_launch(const FwdArgs& a, cudaStream_t s) {
  constexpr int B = G < 128 ? 128 : G, rows = B / G;
  return launch_pdl(rn_fwd_kernel<XT, OT, G, PER, ANY>, (unsigned)((a.M + rows - 1) / rows), B, 0,
                    s, 1, a);
}
template <typename XT, typename OT, bool ANY>
cudaError_t fwd_typed(const FwdArgs& a, bool rows, cudaStream_t s) {
  const int64_t C = rows ? a.N + (ANY ? 7 : 0) : INT64_MAX;
  // Up to 32 elements a thread: as few warps a row as hold it, for many rows in flight (16384 x
  // 2880: 87 us). Too few rows to fill the GPU that way: as many threads as the row feeds, which
  // is there sooner.
  const bool many = a.M >= (int64_t)std::max(device_sms(), 1) * 2;
  if (C <= 32 * 8) return fwd_launch<XT, OT, ANY, 32, 1>(a, s);
  if (many) {
    if (C <= 32 * 16) return fwd_launch<XT, OT, ANY, 32, 2>(a, s);
    if (C <= 128 * 8) return fwd_launch<XT, OT, ANY, 128, 1>(a, s);
    if (C <= 128 * 16) return fwd_launch<XT, OT, ANY, 128, 2>(a, s);
    // a row just below a power of two needs seven columns more off the boundaries
    if constexpr (ANY)
      if (C <= 160 * 16) return fwd_launch<XT, OT, ANY, 160, 2>(a, s);
    if (C <= 128 * 24) return fwd_launch<XT, OT, ANY, 128, 3>(a, s);
    if (C <= 128 * 32) return fwd_launch<XT, OT, ANY, 128, 4>(a, s);
    if constexpr (ANY)
      if (C <= 160 * 32) return fwd_launch<XT, OT, ANY, 160, 4>(a, s);
    if (C <= 256 * 32) return fwd_launch<XT, OT, ANY, 256, 4>(a, s);
  }
  if (C <= 256 * 8) return fwd_launch<XT, OT, ANY, 256, 1>(a, s);
  if (C <= 512 * 8) return fwd_launch<XT, OT, ANY, 512, 1>(a, s);
  if (C <= 1024 * 8) return fwd_launch<XT, OT, ANY, 1024, 1>(a, s);
  if (C <= 1024 * 16) return fwd_launch<XT, OT, ANY, 1024, 2>(a, s);
  const int grid = (int)std::min<int64_t>(a.M, (int64_t)std::max(device_sms(), 1) * 2);
  return launch_pdl(rn_fwd_any_kernel<XT, OT>, grid, 1024, 0, s, 1, a);
}

// The partial sums that a backward kernel leaves.
struct Parts {
  int n = 0;
  bool done = false;     // a single block has written the weights' gradients
  bool shifted = false;  // block b's lie like row b in its vectors
};
// Rows of the ring: as many as leave room for two blocks an SM (where the registers hold only one:
// for that one), up to four; at least one.
template <typename XT, typename OT, int G, int PER>
constexpr int ring_rows() {
  constexpr int bytes = units<XT, OT>() * PER * block_of(G) * 16;
  constexpr int n = (G >= 512 ? 200 : 112) * 1024 / bytes;
  return n > 4 ? 4 : n < 1 ? 1 : n;
}
template <typename XT, typename OT, bool ANY, int G, int PER>
cudaError_t bwd_launch(const BwdArgs& a, Parts& parts, cudaStream_t s) {
  constexpr int B = block_of(G), GROUPS = B / G, S = ring_rows<XT, OT, G, PER>();
  constexpr int smem = (S * PER * B + (ANY ? S * GROUPS : 0)) * units<XT, OT>() * 16;
  static_assert(smem <= 208 * 1024, "shared memory of a block");
  auto kern = rn_bwd_kernel<XT, OT, G, PER, S, ANY>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem);
  if (e != cudaSuccess) return e;
  // as many blocks as fit at once, each a row of partials
  static DeviceCache cache;
  const int per_sm = std::max(1, cache.get(current_device(), [&] {
    return blocks_per_sm(reinterpret_cast<const void*>(kern), B, smem);
  }));
  const int64_t fit = std::min<int64_t>((int64_t)std::max(device_sms(), 1) * per_sm, kMaxParts);
  parts.n = (int)std::max<int64_t>(1, std::min<int64_t>((a.M + GROUPS - 1) / GROUPS, fit));
  if (ANY && (int64_t)parts.n * GROUPS < a.M)  // rows of a group lie alike
    parts.n = std::max(parts.n * GROUPS / 8 * 8, 8) / GROUPS;
  parts.done = parts.n == 1;
  parts.shifted = ANY && GROUPS == 1;
  return launch_pdl(kern, parts.n, B, smem, s, 1, a);
}
template <typename XT, typename OT, bool ANY>
cudaError_t bwd_typed(const BwdArgs& a, bool rows, Parts& parts, cudaStream_t s) {
  const int64_t C = rows ? a.N : INT64_MAX;
  if (C <= 32 * 8) return bwd_launch<XT, OT, ANY, 32, 1>(a, parts, s);
  if (C <= 32 * 16) return bwd_launch<XT, OT, ANY, 32, 2>(a, parts, s);
  if (C <= 128 * 8) return bwd_launch<XT, OT, ANY, 128, 1>(a, parts, s);
  if (C <= 256 * 8) return bwd_launch<XT, OT, ANY, 256, 1>(a, parts, s);
  if (C <= 256 * 16) return bwd_launch<XT, OT, ANY, 256, 2>(a, parts, s);
  if (C <= 512 * 16) return bwd_launch<XT, OT, ANY, 512, 2>(a, parts, s);
  if constexpr (sizeof(OT) == 2)
    if (C <= 512 * 32) return bwd_launch<XT, OT, ANY, 512, 4>(a, parts, s);
  parts.n = (int)std::min<int64_t>(
      a.M, std::min<int64_t>((int64_t)std::max(device_sms(), 1) * 2, kMaxParts));
  return launch_pdl(rn_bwd_any_kernel<XT, OT>, parts.n, 1024, 0, s, 1, a);
}

bool on(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
int size_of(int32_t dtype) { return dtype == MOE_DT_FP32 ? 4 : 2; }

// Calls fn with values of the stream's and the branch's type.
template <class F>
cudaError_t typed(int32_t xd, int32_t od, F&& fn) {
  if (xd == MOE_DT_BF16) return fn(__nv_bfloat16(), __nv_bfloat16());
  if (od == MOE_DT_BF16) return fn(float(), __nv_bfloat16());
  return fn(float(), float());
}

moe_status_t check_types(int64_t M, int64_t N, int32_t xd, int32_t od, int32_t wd) {
  if (M < 0 || N < 1) return fail(MOE_ERR_INVALID_ARG, "M must be >= 0 and N >= 1");
  if (N > INT32_MAX || M > INT32_MAX) return fail(MOE_ERR_UNSUPPORTED, "M or N too large");
  for (int32_t d : {xd, od, wd})
    if (d != MOE_DT_BF16 && d != MOE_DT_FP32) return fail(MOE_ERR_INVALID_ARG, "unknown dtype");
  if (xd == MOE_DT_BF16 && od == MOE_DT_FP32)
    return fail(MOE_ERR_UNSUPPORTED, "a bf16 stream takes bf16 branches");
  if (od == MOE_DT_FP32 && wd == MOE_DT_BF16)
    return fail(MOE_ERR_UNSUPPORTED, "fp32 branches take fp32 weights");
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_residual_norm_fwd(const void* x, int64_t ldx, const void* o, int64_t ldo,
                                   const void* post_weight, const float* gate,
                                   const void* weight, void* x_new, int64_t ldxn, void* h,
                                   int64_t ldh, float* rstd_post, float* rstd, int64_t M,
                                   int64_t N, float scale, int32_t post_norm, float eps,
                                   int32_t x_dtype, int32_t o_dtype, int32_t w_dtype,
                                   moe_stream_t stream) {
  moe_status_t st = check_types(M, N, x_dtype, o_dtype, w_dtype);
  if (st != MOE_OK) return st;
  if (!(eps >= 0.f)) return fail(MOE_ERR_INVALID_ARG, "eps must be >= 0");
  if (M == 0) return MOE_OK;  // empty tensors' pointers may be NULL
  if ((o != nullptr) != (x_new != nullptr))
    return fail(MOE_ERR_INVALID_ARG, "o and x_new go together");
  if (!o && (post_weight || gate || post_norm))
    return fail(MOE_ERR_INVALID_ARG, "post_weight, gate and post_norm need a branch");
  if (!h && weight) return fail(MOE_ERR_INVALID_ARG, "weight needs h");
  if (!o && !h) return fail(MOE_ERR_INVALID_ARG, "neither a branch nor h");
  if (ldx < N || (o && (ldo < N || ldxn < N)) || (h && ldh < N))
    return fail(MOE_ERR_INVALID_ARG, "row strides must be >= N");
  if (x_new == x && x_new && ldxn != ldx)
    return fail(MOE_ERR_INVALID_ARG, "x_new is x, with another row stride");
  if (h == o && h && ldh != ldo)
    return fail(MOE_ERR_INVALID_ARG, "h is o, with another row stride");
  const int xb = size_of(x_dtype), ob = size_of(o_dtype), wb = size_of(w_dtype);
  const Span sx = span(x, N, ldx, xb), so = span(o, N, ldo, ob);
  const Span sn = span(x_new, N, ldxn, xb), sh = span(h, N, ldh, ob);
  if (spoils(sn, sx, M) || spoils(sn, so, M) || spoils(sh, sx, M) || spoils(sh, so, M) ||
      spoils(sh, sn, M) || (h && h == x_new))
    return fail(MOE_ERR_INVALID_ARG, "an output shares memory with another tensor's other rows");
  if (!on(x, xb) || !on(x_new, xb) || !on(o, ob) || !on(h, ob) || !on(post_weight, wb) ||
      !on(weight, wb) || !on(gate, 4) || !on(rstd_post, 4) || !on(rstd, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (!x) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
  const int w32 = w_dtype == MOE_DT_FP32;
  const FwdArgs a = {x, o, x_new, h, ldx, ldo, ldxn, ldh, M, N,
                     {post_weight, (int16_t)w32, on(post_weight, 16)},
                     {weight, (int16_t)w32, on(weight, 16)}, gate, rstd_post, rstd, scale, eps,
                     post_norm != 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Places at;
  at.add(x, ldx, xb);
  at.add(x_new, ldxn, xb);
  at.add(o, ldo, ob);
  at.add(h, ldh, ob);
  const bool any = !(at.aligned && N % 8 == 0 && a.wp.vec && a.w.vec);
  const cudaError_t e = typed(x_dtype, o_dtype, [&](auto xt, auto ot) {
    using XT = decltype(xt);
    using OT = decltype(ot);
    return any ? fwd_typed<XT, OT, true>(a, at.same, s) : fwd_typed<XT, OT, false>(a, true, s);
  });
  count_launch(s, MOE_K_RESIDUAL_NORM_FWD);
  if (e != cudaSuccess) return cuda_fail(e, "residual norm forward launch");
  return MOE_OK;
}

size_t moe_residual_norm_workspace(int64_t M, int64_t N) {
  if (M < 0 || N < 1 || M > INT32_MAX || N > INT32_MAX) {
    fail(MOE_ERR_INVALID_ARG, "M must be in [0, 2^31) and N in [1, 2^31)");
    return 0;
  }
  return (size_t)std::max<int64_t>(1, std::min<int64_t>(M, kMaxParts)) * 2 * part_pitch(N) *
         sizeof(float);
}

moe_status_t moe_residual_norm_bwd(const void* dh, int64_t lddh, const void* dx_new,
                                   int64_t lddxn, const void* x_new, int64_t ldxn, const void* o,
                                   int64_t ldo, const void* post_weight, const float* gate,
                                   const void* weight, const float* rstd_post, const float* rstd,
                                   void* dx, int64_t lddx, void* d_o, int64_t lddo,
                                   void* d_post_weight, void* d_weight, float* d_gate, int64_t M,
                                   int64_t N, float scale, int32_t post_norm, int32_t x_dtype,
                                   int32_t o_dtype, int32_t w_dtype, void* ws, size_t ws_bytes,
                                   moe_stream_t stream) {
  moe_status_t st = check_types(M, N, x_dtype, o_dtype, w_dtype);
  if (st != MOE_OK) return st;
  const bool weights = d_weight || d_post_weight;
  if (M > 0) {  // empty tensors' pointers may be NULL
    if (!dh && !dx_new) return fail(MOE_ERR_INVALID_ARG, "neither dh nor dx_new");
    if (!dh && (weight || d_weight))
      return fail(MOE_ERR_INVALID_ARG, "weight and d_weight need dh");
    if (dh && (!x_new || !rstd)) return fail(MOE_ERR_INVALID_ARG, "dh needs x_new and rstd");
    if (!o && (d_o || d_post_weight || d_gate || post_weight || gate || post_norm))
      return fail(MOE_ERR_INVALID_ARG, "post_weight, gate, post_norm and gradients need a branch");
    if (post_norm && !rstd_post) return fail(MOE_ERR_INVALID_ARG, "post_norm needs rstd_post");
    if (d_gate && !gate) return fail(MOE_ERR_INVALID_ARG, "d_gate needs a gate");
    if (!dx && !d_o && !weights && !d_gate) return fail(MOE_ERR_INVALID_ARG, "nothing to write");
    if ((dh && (lddh < N || ldxn < N)) || (dx_new && lddxn < N) || (o && ldo < N) ||
        (dx && lddx < N) || (d_o && lddo < N))
      return fail(MOE_ERR_INVALID_ARG, "row strides must be >= N");
    if ((dx && dx == dx_new && lddx != lddxn) || (d_o && d_o == dh && lddo != lddh) ||
        (d_o && d_o == o && lddo != ldo))
      return fail(MOE_ERR_INVALID_ARG, "an output is an input, with another row stride");
  }
  if (d_post_weight && !post_weight)
    return fail(MOE_ERR_INVALID_ARG, "d_post_weight needs post_weight");
  const int xb = size_of(x_dtype), ob = size_of(o_dtype), wb = size_of(w_dtype);
  if (!on(dh, ob) || !on(dx_new, xb) || !on(x_new, xb) || !on(o, ob) || !on(dx, xb) ||
      !on(d_o, ob) || !on(post_weight, wb) || !on(weight, wb) || !on(d_post_weight, wb) ||
      !on(d_weight, wb) || !on(gate, 4) || !on(rstd_post, 4) || !on(rstd, 4) || !on(d_gate, 4))
    return fail(MOE_ERR_INVALID_ARG, "tensors must be aligned to their elements");
  if (weights) {
    if (!ws || !on(ws, 16))
      return fail(MOE_ERR_INVALID_ARG, "ws must be non-NULL and 16-byte aligned");
    if (ws_bytes < moe_residual_norm_workspace(M, N))
      return fail(MOE_ERR_WORKSPACE, "ws_bytes=%zu < required %zu", ws_bytes,
                  moe_residual_norm_workspace(M, N));
  }
  if (M > 0) {
    const Span in[4] = {span(dh, N, lddh, ob), span(dx_new, N, lddxn, xb),
                        span(dh ? x_new : nullptr, N, ldxn, xb), span(o, N, ldo, ob)};
    const Span sx = span(dx, N, lddx, xb), so = span(d_o, N, lddo, ob);
    bool bad = spoils(so, sx, M) || (dx && dx == d_o);
    for (const Span& i : in) bad = bad || spoils(sx, i, M) || spoils(so, i, M);
    if (bad)
      return fail(MOE_ERR_INVALID_ARG, "an output shares memory with another tensor's other rows");
  }
  if (M == 0 && !weights) return MOE_OK;
  const int w32 = w_dtype == MOE_DT_FP32;
  float* part = weights ? static_cast<float*>(ws) : nullptr;
  const BwdArgs a = {dh, dx_new, x_new, o, dx, d_o, lddh, lddxn, ldxn, ldo, lddx, lddo, M, N,
                     {post_weight, (int16_t)w32, on(post_weight, 16)},
                     {weight, (int16_t)w32, on(weight, 16)}, gate, rstd_post, rstd, d_gate, scale,
                     post_norm != 0, part, d_weight, d_post_weight, w32};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  Parts parts;
  Places at;
  if (M > 0) {
    if (dh) {
      at.add(dh, lddh, ob);
      at.add(x_new, ldxn, xb);
    }
    at.add(dx_new, lddxn, xb);
    at.add(dx, lddx, xb);
    at.add(o, ldo, ob);
    at.add(d_o, lddo, ob);
    const bool any = !(at.aligned && N % 8 == 0 && a.wp.vec && a.w.vec);
    e = typed(x_dtype, o_dtype, [&](auto xt, auto ot) {
      using XT = decltype(xt);
      using OT = decltype(ot);
      return any ? bwd_typed<XT, OT, true>(a, at.same, parts, s)
                 : bwd_typed<XT, OT, false>(a, true, parts, s);
    });
    count_launch(s, MOE_K_RESIDUAL_NORM_BWD);
    if (e != cudaSuccess) return cuda_fail(e, "residual norm backward launch");
  }  // no rows: no partials, the sums are zero
  if (weights && !parts.done) {
    const unsigned grid = (unsigned)((2 * N + 31) / 32);
    const uint32_t place = parts.shifted ? (uint32_t)at.place : 0u;
    const uint32_t pitch = parts.shifted ? (uint32_t)at.pitch : 0u;
    if (w32)
      e = launch_pdl(rn_colsum_kernel<float>, grid, 1024, 0, s, 1, (const float*)part, parts.n, N,
                     static_cast<float*>(d_weight), static_cast<float*>(d_post_weight), place,
                     pitch);
    else
      e = launch_pdl(rn_colsum_kernel<__nv_bfloat16>, grid, 1024, 0, s, 1, (const float*)part,
                     parts.n, N, static_cast<__nv_bfloat16*>(d_weight),
                     static_cast<__nv_bfloat16*>(d_post_weight), place, pitch);
    count_launch(s, MOE_K_RESIDUAL_NORM_REDUCE);
    if (e != cudaSuccess) return cuda_fail(e, "residual norm reduction launch");
  }
  return MOE_OK;
}

}  // extern "C"
