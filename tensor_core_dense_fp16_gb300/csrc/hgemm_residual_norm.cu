// hgemm_residual_norm.cu — the norms around a block with its gate and the
// residual's scale, forward and backward (the formulas are in hgemm.h). Both
// are bound by memory: forward reads 4 bytes per value and writes 4, backward
// reads 8 and writes 4. Measured: forward 16384×4096, RMS norms, 80 us, layer
// norms 88 (79 at a copy's rate); backward 16384×8192, RMS norms, 248 us (237).
#include <atomic>
#include <type_traits>

#include <cuda_fp16.h>

#include "debug.cuh"
#include "hgemm.h"
#include "internal.h"
#include "kernel_common.cuh"
#include "ptx.cuh"
#include "row_sums.cuh"

namespace hg {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float half_or(const uint16_t* p, int64_t i, float otherwise) {
  return p ? half_at(p, i) : otherwise;
}

// ------------------------------------------------------------------ forward

__device__ __forceinline__ float pair_sum(f32x2 v) {
  float lo, hi;
  unpair(v, lo, hi);
  return lo + hi;
}

// What a warp knows of its row's values: their mean (RMS: 0) and the sum of
// the squares around it.
struct Part {
  float mean, sq;
};

// The values a thread holds, 8·NV in pairs; those past the row's end are 0.
// VEC: the row in 16-byte pieces; otherwise value by value, neighbouring
// threads on neighbouring values.
template <int G, int NV, bool VEC>
struct RowPiece {
  int t, D;
  // the column of value k of piece j
  __device__ int col(int j, int k) const { return VEC ? (t + j * G) * 8 + k : (8 * j + k) * G + t; }
  __device__ bool in(int j, int k) const { return col(j, VEC ? 0 : k) < D; }
  // How many of the row's values this thread's warp holds.
  __device__ int of_warp() const {
    int n = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < (VEC ? 1 : 8); ++k) n += __popc(__ballot_sync(0xffffffffu, in(j, k)));
    return VEC ? 8 * n : n;
  }
  __device__ uint4 load(const uint16_t* p, int j) const {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if constexpr (VEC) {
      const int c = col(j, 0);
      if (c < D && dbg_row(p + c, c, 8, D, 16)) v = load16(p + c);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = in(j, k) ? p[col(j, k)] : 0u;
      v = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
    return v;
  }
  __device__ void store(uint16_t* p, int j, const float (&f)[8]) const {
    const uint4 v = pack8f(f);
    if constexpr (VEC) {
      const int c = col(j, 0);
      if (c < D && dbg_row(p + c, c, 8, D, 16)) *reinterpret_cast<uint4*>(p + c) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (in(j, k)) p[col(j, k)] = static_cast<uint16_t>(w[k / 2] >> (16 * (k & 1)));
    }
  }
};

// μ and ρ of a row from the moments of the G threads that hold it; `n` of its
// values lie in this warp, counts[w] in warp w. A layer norm's squares are
// summed around each warp's own mean, and the warps' joined by the distances
// of their means: Σ(v − μ)² = Σ_w [Σ(v − μ_w)² + n_w·(μ_w − μ)²], which keeps
// its digits in a row far from zero and takes one exchange between the warps
// where a second pass around the row's mean takes two.
template <int G, int NV, bool VEC>
__device__ __forceinline__ void row_moments(bool layer, const RowPiece<G, NV, VEC>& piece, float eps, float n,
                                            const float* counts, Part* parts, const float (&v)[NV][8], float& mu,
                                            float& rho) {
  Part p{0.f, 0.f};
  if (layer) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[j][k];
    p.mean = n > 0.f ? warp_sum(s) / n : 0.f;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float c = VEC || piece.in(j, k) ? v[j][k] - p.mean : 0.f;
      sq = fmaf(c, c, sq);
    }
    if (piece.in(j, 0)) p.sq += sq;
  }
  p.sq = warp_sum(p.sq);
  const float inv = 1.f / static_cast<float>(piece.D);
  mu = p.mean;
  if constexpr (G > 32) {
    if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = p;
    __syncthreads();
    float sum = 0.f, total = 0.f;
    if (layer) {
#pragma unroll
      for (int w = 0; w < G / 32; ++w) sum = fmaf(counts[w], parts[w].mean, sum);
      mu = sum * inv;
#pragma unroll
      for (int w = 0; w < G / 32; ++w) {
        const Part q = parts[w];
        total += fmaf(counts[w] * (q.mean - mu), q.mean - mu, q.sq);
      }
    } else {
#pragma unroll
      for (int w = 0; w < G / 32; ++w) total += parts[w].sq;
    }
    p.sq = total;
  }
  rho = rsqrtf(p.sq * inv + eps);
}

// G threads per row, which they hold in registers; one read and one write.
// A block per row, or per four rows of a warp each. (At least 768 threads to an
// SM where a thread holds 32 values: 16384 rows of 8192, RMS norms: 169 us, and
// 194 with the registers that the compiler takes without the bound.)
//
// `ahead`, or 0: a row's first thread asks L2 for the rows that come when this
// wave of blocks has ended, so that memory is busy while blocks compute: layer
// norms 16384×4096 92 us without, 88 with it, 101 two waves ahead; 16384×8192 204
// and 200, RMS norms 166 and 158. Short rows of RMS norms have no time to fill
// (16384×4096 80.2 us without, 81.3 with it).
constexpr int kResident = 768;
template <int G>
constexpr int kRowsThreads = G < 64 ? 128 : G;
template <int G, int NV, bool VEC>
__global__ void __launch_bounds__(kRowsThreads<G>, NV == 4 && G < 512 ? kResident / kRowsThreads<G> : 1)
    residual_norm_rows_kernel(const ResidualNormArgs a, const int ahead) {
  constexpr int THREADS = kRowsThreads<G>;
  __shared__ Part parts[2][THREADS / 32];
  __shared__ float counts[THREADS / 32];
  const RowPiece<G, NV, VEC> piece{static_cast<int>(threadIdx.x % G), static_cast<int>(a.D)};
  const int64_t m = static_cast<int64_t>(blockIdx.x) * (THREADS / G) + threadIdx.x / G;
  float n = 0.f;
  if (a.post == HGEMM_NORM_LAYER || a.pre == HGEMM_NORM_LAYER) {
    n = static_cast<float>(piece.of_warp());
    if ((threadIdx.x & 31) == 0) counts[threadIdx.x >> 5] = n;  // (read behind the exchanges' barriers)
  }
  grid_dependency_wait();
  grid_launch_dependents();
  if (G < 64 && m >= a.M) return;  // whole warps; larger groups have a block of their own
  if (VEC && NV == 4 && piece.t == 0 && ahead > 0 && m + ahead < a.M) {
    bulk_prefetch(a.y + (m + ahead) * a.ldy, static_cast<uint32_t>(a.D) * 2u);
    bulk_prefetch(a.x + (m + ahead) * a.ldx, static_cast<uint32_t>(a.D) * 2u);
  }
  float v[NV][8];                   // y, then z
  uint4 x[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) x[j] = piece.load(a.y + m * a.ldy, j);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    unpack8(x[j], v[j]);
    x[j] = piece.load(a.x + m * a.ldx, j);
  }
  float my = 0.f, ry = 1.f, mz = 0.f, rz = 1.f;
  if (a.post) row_moments(a.post == HGEMM_NORM_LAYER, piece, a.eps, n, counts, parts[0], v, my, ry);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float f[8];
    if (a.post) {
      unpack8(piece.load(a.post_gamma, j), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = (v[j][k] - my) * ry * f[k];
      if (a.post_beta) {
        unpack8(piece.load(a.post_beta, j), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] += f[k];
      }
    }
    if (a.gate) {
      unpack8(piece.load(a.gate, j), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= f[k];
    }
    unpack8(x[j], f);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] = fmaf(a.alpha, f[k], v[j][k]);
    piece.store(a.z + m * a.ldz, j, v[j]);
  }
  if (a.pre) {
    row_moments(a.pre == HGEMM_NORM_LAYER, piece, a.eps, n, counts, parts[1], v, mz, rz);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
      unpack8(piece.load(a.pre_gamma, j), f);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = (v[j][k] - mz) * rz * f[k];
      if (a.pre_beta) {
        unpack8(piece.load(a.pre_beta, j), f);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] += f[k];
      }
      piece.store(a.h + m * a.ldh, j, v[j]);
    }
  }
  if (piece.t == 0 && a.stats && HG_DBG_INDEX(m, a.M)) {
    if (a.post) a.stats[m] = my, a.stats[a.M + m] = ry;
    if (a.pre) a.stats[2 * a.M + m] = mz, a.stats[3 * a.M + m] = rz;
  }
}

// Rows too long for registers: a block per row, which it reads once per sum
// (from L1 or L2 after the first).

// μ and ρ of a row's values v(d), d = threadIdx.x, + kThreads, ...
template <typename Value>
__device__ __forceinline__ void long_row_moments(int kind, int64_t D, float eps, float* s, Value v, float& mu, float& rho) {
  const float n = static_cast<float>(D);
  mu = 0.f;
  if (kind == HGEMM_NORM_LAYER) {
    float sum = 0.f;
    for (int64_t d = threadIdx.x; d < D; d += kThreads) sum += v(d);
    mu = group_sum<kThreads>(sum, s) / n;
  }
  float sq = 0.f;
  for (int64_t d = threadIdx.x; d < D; d += kThreads) {
    const float c = v(d) - mu;
    sq = fmaf(c, c, sq);
  }
  rho = rsqrtf(group_sum<kThreads>(sq, s) / n + eps);
}

__global__ void __launch_bounds__(kThreads) residual_norm_long_kernel(const ResidualNormArgs a) {
  __shared__ float s[kThreads / 32];
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    if (!HG_DBG_INDEX(m, a.M)) return;
    const uint16_t *x = a.x + m * a.ldx, *y = a.y + m * a.ldy;
    float my = 0.f, ry = 1.f, mz = 0.f, rz = 1.f;
    if (a.post) long_row_moments(a.post, a.D, a.eps, s, [&](int64_t d) { return half_at(y, d); }, my, ry);
    auto z = [&](int64_t d) {
      float n = half_at(y, d);
      if (a.post) n = fmaf((n - my) * ry, half_at(a.post_gamma, d), half_or(a.post_beta, d, 0.f));
      return fmaf(a.alpha, half_at(x, d), n * half_or(a.gate, d, 1.f));
    };
    if (a.pre) long_row_moments(a.pre, a.D, a.eps, s, z, mz, rz);
    __syncthreads();  // (Z may be X and H may be Y) the row has been read
    for (int64_t d = threadIdx.x; d < a.D; d += kThreads) {
      const float v = z(d);
      a.z[m * a.ldz + d] = __half_as_ushort(__float2half_rn(v));
      if (a.pre)
        a.h[m * a.ldh + d] = __half_as_ushort(
            __float2half_rn(fmaf((v - mz) * rz, half_at(a.pre_gamma, d), half_or(a.pre_beta, d, 0.f))));
    }
    if (threadIdx.x == 0 && a.stats) {
      if (a.post) a.stats[m] = my, a.stats[a.M + m] = ry;
      if (a.pre) a.stats[2 * a.M + m] = mz, a.stats[3 * a.M + m] = rz;
    }
  }
}

// ----------------------------------------------------------------- backward

// Persistent CTAs of 512 threads, one per SM, in groups of G threads; group j
// of a CTA owns a row at a time. Rows arrive by bulk copies, several ahead, in
// a ring per group: dZ, dH, Z and Y, as far as there are any. A thread owns
// the same 16 columns of every row, so the column sums add up in its
// registers; at the end the groups of a CTA are added in order through shared
// memory and the CTA writes one partial sum of each.
//
// Per row: pass 1 gives every sum along the row, one exchange between the
// group's warps, pass 2 gives dX, dY and the columns' terms. That one exchange
// is enough because dz is linear in a1 and a2: with t = dZ + ρ_z·g,
// Σ w·dz = Σ w·t − ρ_z·(a1·Σw + a2·Σ w·ẑ), and the same with w·ŷ for w. Pass 1
// of a row runs before pass 2 of the row before it, so that the exchange has
// the time of a pass. Both passes read shared memory, which keeps the
// registers for the column sums. The barrier of the exchange also frees the
// stage of the row before: every thread of the group has finished its pass 2
// by then, and a row is copied into it.
//
// FULL: a layer norm, or a beta's gradient, is among what is wanted: four
// column sums and the sums along the row that only these need. RMS norms
// without betas do without, which leaves registers to run both passes in.
struct RingPlan {
  uint32_t dz, dh, z, y;  // where a row of each lies in a stage
  uint32_t stage_bytes;
  int stages;
  bool need_y;            // the norm behind the block or the gate's gradient reads Y
  bool empty;             // nothing to copy: neither dZ nor dH, nor Y
};

template <int G_>
struct RingCfg {
  static constexpr int G = G_, NV = 2;
  static constexpr int THREADS = 512;
  static constexpr int GROUPS = THREADS / G;
  static constexpr int WARPS = G / 32;  // per group
  static constexpr int MAX_STAGES = 8;
  static constexpr int RING_BYTES = 192 * 1024;  // of the CTA
  static constexpr int OFF_W = RING_BYTES;       // FULL: gate·post_gamma of up to 8192 columns,
  static constexpr bool SHARED_GAMMA = 2 * G <= THREADS;
  static constexpr int OFF_GAMMA = OFF_W + G * 8 * NV * 4;  // with pre_gamma behind it where there is room
  static constexpr int OFF_BAR = OFF_W + THREADS * 8 * NV * 4;
  static constexpr int OFF_EXCHANGE = OFF_BAR + GROUPS * MAX_STAGES * 8;
  static constexpr int OFF_MISC = OFF_EXCHANGE + 2 * (THREADS / 32) * 32;  // two buffers of eight sums per warp
  static constexpr int SMEM_BYTES = OFF_MISC + 16;
  static_assert(SMEM_BYTES <= 232448, "fits a CTA");
  static_assert(THREADS * 8 * NV * 4 * 4 <= RING_BYTES, "the groups' sums fit the ring");
};

// N sums (4 or 8) over a warp: while more than one is left, a lane sends the
// half of them that its partner goes on with; 9 shuffles for eight. Lane l
// leaves with the sum of v[l % N] over all lanes.
template <int N>
__device__ __forceinline__ float warp_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const float mine = upper ? v[i + o] : v[i], other = upper ? v[i] : v[i + o];
      v[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
    }
  }
  float r = v[0];
#pragma unroll
  for (int o = N; o < 32; o <<= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// A row's statistics (mean and 1/σ of Y, then of Z), and where it lies in the
// ring. LANES: one to a lane (lane % 4), handed out by a shuffle, and an offset
// in place of an address: two registers in place of six for each of the three
// rows under way.
template <bool LANES>
struct RingRow {
  float stat[LANES ? 1 : 4];
  std::conditional_t<LANES, uint32_t, const uint8_t*> at;
  __device__ float of(int i) const {
    if constexpr (LANES)
      return __shfl_sync(0xffffffffu, stat[0], i);
    else
      return stat[i];
  }
};

template <int G, bool POST, bool PRE, bool FULL>
__global__ void __launch_bounds__(512, 1) residual_norm_ring_kernel(const ResidualNormBackArgs a, const RingPlan plan) {
  using Cfg = RingCfg<G>;
  constexpr int NV = Cfg::NV;
  constexpr int SUMS = FULL ? 8 : 4;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  const int group = threadIdx.x / G, t = threadIdx.x % G;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int D = static_cast<int>(a.D), stages = plan.stages;
  const uint32_t row_bytes = static_cast<uint32_t>(D) * 2u;
  uint8_t* ring = ring_smem + static_cast<uint32_t>(group * stages) * plan.stage_bytes;
  const uint32_t ring_addr = smem_u32(ring);
  const uint32_t bar0 = smem_u32(ring_smem + Cfg::OFF_BAR) + static_cast<uint32_t>(group * Cfg::MAX_STAGES * 8);
  float* exchange = reinterpret_cast<float*>(ring_smem + Cfg::OFF_EXCHANGE);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(ring_smem + Cfg::OFF_MISC);
  const Watchdog wd{abort_flag, a.status, a.timeout_ns};

  if (threadIdx.x == 0) *abort_flag = 0;
  if (t == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(bar0 + 8u * i, 1);
    fence_barrier_init();
  }
  __syncthreads();
  grid_dependency_wait();
  grid_launch_dependents();

  const int64_t first = static_cast<int64_t>(blockIdx.x) * Cfg::GROUPS + group;
  const int64_t step = static_cast<int64_t>(gridDim.x) * Cfg::GROUPS;
  // With all sums of both norms the arithmetic is what a row waits for: the
  // first lanes of four warps issue its copies, an operand each, since one
  // thread's hold its warp up, and then the group (layer norms, 16384×4096: 191
  // µs by one thread, 168 by four). Elsewhere memory is, and one thread is
  // faster (RMS norms 122 and 124, one layer norm 123 and 136), with the
  // statistics in registers.
  constexpr bool BUSY = FULL && POST && PRE;
  constexpr int COPIERS = !BUSY ? 1 : Cfg::WARPS < 4 ? Cfg::WARPS : 4;
  const bool copier = lane == 0 && t < 32 * COPIERS;
  int copied = 0;  // rows that this thread has issued copies of
  auto copy_row = [&](int64_t m, int stage) {
    if (plan.empty) return;
    ++copied;
    const uint32_t bar = bar0 + 8u * stage, dst = ring_addr + static_cast<uint32_t>(stage) * plan.stage_bytes;
    const int who = COPIERS == 1 ? 0 : t / 32;
    if (t == 0 && !(a.inject == 1 && copied == 1))  // testing aid: withhold one arrival
      mbar_arrive_expect_tx(bar, plan.stage_bytes);
    if (a.dz && who == 0) bulk_load(dst + plan.dz, a.dz + m * a.lddz, row_bytes, bar);
    if (PRE) {
      if (who == 1 % COPIERS) bulk_load(dst + plan.dh, a.dh + m * a.lddh, row_bytes, bar);
      if (who == 2 % COPIERS) bulk_load(dst + plan.z, a.z + m * a.ldz, row_bytes, bar);
    }
    if ((POST || plan.need_y) && who == 3 % COPIERS) bulk_load(dst + plan.y, a.y + m * a.ldy, row_bytes, bar);
  };
  if (copier)
    for (int i = 0; i < stages - 1; ++i)
      if (first + i * step < a.M) copy_row(first + i * step, i);

  // w = gate·post_gamma, and the norm in front's gamma; the sums dz·ŷ, dz,
  // dH·ẑ and dH of this thread's columns
  // (FULL keeps w in shared memory, and pre_gamma where there is room for it:
  // its sums leave too few registers. Layer norms, 16384×4096: 207 µs with gamma
  // in registers, 195 this way.)
  constexpr bool SHARED_GAMMA = FULL && PRE && Cfg::SHARED_GAMMA;
  f32x2 w[FULL ? 1 : NV][4];
  uint4 gamma[NV];
  ulonglong2* shared_w = reinterpret_cast<ulonglong2*>(ring_smem + Cfg::OFF_W);
  ulonglong2* shared_gamma = reinterpret_cast<ulonglong2*>(ring_smem + Cfg::OFF_GAMMA);
  f32x2 s1[NV][4], s0[NV][4], t1[NV][4], t0[NV][4];
  float sum_w = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * G) * 8;
    gamma[i] = make_uint4(0u, 0u, 0u, 0u);
    f32x2 v[4], f[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = pair_of(c < D ? 1.f : 0.f);
      s1[i][k] = s0[i][k] = t1[i][k] = t0[i][k] = 0;  // a pair of +0
    }
    if (c < D) {
      if (PRE && dbg_row(a.pre_gamma + c, c, 8, D, 16)) gamma[i] = load16(a.pre_gamma + c);
      if (a.gate && dbg_row(a.gate + c, c, 8, D, 16)) unpack8(load16(a.gate + c), v);
      if (POST && dbg_row(a.post_gamma + c, c, 8, D, 16)) {
        unpack8(load16(a.post_gamma + c), f);
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = mul2(v[k], f[k]);
      }
    }
    if constexpr (FULL) {
#pragma unroll
      for (int k = 0; k < 4; ++k) sum_w += pair_sum(v[k]);
      if (group == 0) {
        shared_w[(t + i * G) * 2] = make_ulonglong2(v[0], v[1]);
        shared_w[(t + i * G) * 2 + 1] = make_ulonglong2(v[2], v[3]);
        if constexpr (SHARED_GAMMA) {
          unpack8(gamma[i], f);
          shared_gamma[(t + i * G) * 2] = make_ulonglong2(f[0], f[1]);
          shared_gamma[(t + i * G) * 2 + 1] = make_ulonglong2(f[2], f[3]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) w[i][k] = v[k];
    }
  }
  if constexpr (FULL) __syncthreads();
  // w of a thread's piece i
  auto weights = [&](int i, f32x2 (&v)[4]) {
    if constexpr (FULL) {
      const ulonglong2 lo = shared_w[(t + i * G) * 2], hi = shared_w[(t + i * G) * 2 + 1];
      v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = w[i][k];
    }
  };
  auto gammas = [&](int i, f32x2 (&v)[4]) {
    if constexpr (SHARED_GAMMA) {
      const ulonglong2 lo = shared_gamma[(t + i * G) * 2], hi = shared_gamma[(t + i * G) * 2 + 1];
      v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
    } else {
      unpack8(gamma[i], v);
    }
  };

  const float inv_d = 1.f / static_cast<float>(D);
  const bool layer_y = POST && a.post == HGEMM_NORM_LAYER, layer_z = PRE && a.pre == HGEMM_NORM_LAYER;
  int stage = 0;  // of the next row that pass 1 takes
  uint32_t phase = 0;
  auto fetch_stats = [&](int64_t m) {
    RingRow<BUSY> r;
    r.at = 0;
#pragma unroll
    for (int i = 0; i < (BUSY ? 1 : 4); ++i) {
      const int which = BUSY ? lane & 3 : i;
      const bool known = which == 0 ? layer_y : which == 1 ? POST : which == 2 ? layer_z : PRE;
      r.stat[i] = static_cast<float>(which & 1);
      if (known && m < a.M) r.stat[i] = a.stats[which * a.M + m];
    }
    return r;
  };
  auto in_ring = [&](const RingRow<BUSY>& r) -> const uint8_t* {
    if constexpr (BUSY)
      return ring + r.at;
    else
      return r.at;
  };
  // The sums along a row, over this warp's columns, into the exchange:
  // Σ g·ẑ, w·ŷ·t, w·ŷ·ẑ, and FULL Σ g, w·t, w·ẑ, w·ŷ, w.
  auto pass1 = [&](RingRow<BUSY>& r, int flip) {
    // A wait that gives up has raised the abort flag: no more copies are
    // issued, later waits give up at once, and the loop runs out on what the
    // ring holds, so that every thread still reaches every barrier.
    if (!plan.empty) (void)wait_phase(bar0 + 8u * stage, phase, wd, kWdRows);
    if constexpr (BUSY)
      r.at = static_cast<uint32_t>(stage) * plan.stage_bytes;
    else
      r.at = ring + static_cast<uint32_t>(stage) * plan.stage_bytes;
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
    if constexpr (POST || PRE) {
      // (v̂ from the difference: v·ρ − μ·ρ loses its digits in a row far from zero)
      const f32x2 scale_z = pair_of(r.of(3)), shift_z = pair_of(-r.of(2));
      const f32x2 scale_y = pair_of(r.of(1)), shift_y = pair_of(-r.of(0));
      const uint8_t* at = in_ring(r);
      f32x2 p[7] = {0, 0, 0, 0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = t + i * G;
        if (v * 8 < D) {
          f32x2 z[4], tt[4], y[4], g[4];
          if (POST && a.dz) {
            unpack8(reinterpret_cast<const uint4*>(at + plan.dz)[v], tt);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) tt[k] = 0;
          }
          if constexpr (PRE) {
            f32x2 q[4];
            unpack8(reinterpret_cast<const uint4*>(at + plan.z)[v], z);
            unpack8(reinterpret_cast<const uint4*>(at + plan.dh)[v], g);
            gammas(i, q);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (FULL) z[k] = add2(z[k], shift_z);
              z[k] = mul2(z[k], scale_z);
              g[k] = mul2(g[k], q[k]);
              p[0] = fma2(g[k], z[k], p[0]);
              if constexpr (FULL) p[3] = add2(p[3], g[k]);
              tt[k] = fma2(g[k], scale_z, tt[k]);
            }
          }
          if constexpr (POST) {
            f32x2 wv[4];
            weights(i, wv);
            unpack8(reinterpret_cast<const uint4*>(at + plan.y)[v], y);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (FULL) y[k] = add2(y[k], shift_y);
              y[k] = mul2(mul2(y[k], scale_y), wv[k]);  // w·ŷ
              p[1] = fma2(y[k], tt[k], p[1]);
              if constexpr (FULL) p[4] = fma2(wv[k], tt[k], p[4]);
              if constexpr (PRE) {
                p[2] = fma2(y[k], z[k], p[2]);
                if constexpr (FULL) {
                  p[5] = fma2(wv[k], z[k], p[5]);
                  p[6] = add2(p[6], y[k]);
                }
              }
            }
          }
        }
      }
      float sums[SUMS];
#pragma unroll
      for (int i = 0; i < (FULL ? 7 : 3); ++i) sums[i] = pair_sum(p[i]);
      sums[SUMS - 1] = sum_w;
      const float mine = warp_sums(sums);
      if (lane < SUMS) exchange[(flip * (Cfg::THREADS / 32) + warp) * 8 + lane] = mine;
    }
  };

  RingRow<BUSY> row = fetch_stats(first), next = fetch_stats(first + step);
  int flip = 0;
  if (first < a.M) pass1(row, 0);
  for (int64_t m = first; m < a.M; m += step) {
    if constexpr (Cfg::WARPS > 1)
      named_bar_sync(1 + group, G);
    else
      __syncwarp();
    if (copier) {
      // the stage of the row before this one is free: the group is past it
      const int64_t ahead = m + (stages - 1) * step;
      const int into = stage == 0 ? stages - 1 : stage - 1;  // this row's
      if (ahead < a.M && !*abort_flag) copy_row(ahead, into == 0 ? stages - 1 : into - 1);
    }
    float mine = 0.f;
    if constexpr (POST || PRE) {
      const float* ex = exchange + (flip * (Cfg::THREADS / 32) + group * Cfg::WARPS) * 8 + lane % SUMS;
#pragma unroll
      for (int i = 0; i < Cfg::WARPS; ++i) mine += ex[i * 8];
    }
    flip ^= 1;  // the other buffer next: nobody writes this one before everybody has read it
    const RingRow<BUSY> after = fetch_stats(m + 2 * step);
    if (m + step < a.M) pass1(next, flip);

    float sums[SUMS];
    mine *= inv_d;
#pragma unroll
    for (int i = 0; i < SUMS; ++i) sums[i] = __shfl_sync(0xffffffffu, mine, i);
    const float my = row.of(0), ry = row.of(1), mz = row.of(2), rz = row.of(3);
    const uint8_t* at = in_ring(row);
    const float a1 = FULL && layer_z ? sums[SUMS - 5] : 0.f, a2 = sums[0];
    float b1 = 0.f, b2 = sums[1] - rz * (a2 * sums[2]);
    if constexpr (FULL) {
      if (layer_y) b1 = sums[SUMS - 4] - rz * (a1 * sums[SUMS - 1] + a2 * sums[SUMS - 3]);
      b2 -= rz * (a1 * sums[SUMS - 2]);
    }
    // dz = dZ + ρ_z·g + ẑ·k2 + k1;  dY = ρ_y·w·dz + ŷ·l2 + l1
    const f32x2 scale_z = pair_of(rz), shift_z = pair_of(-mz);
    const f32x2 scale_y = pair_of(ry), shift_y = pair_of(-my);
    const f32x2 k1 = pair_of(-rz * a1), k2 = pair_of(-rz * a2);
    const f32x2 l1 = pair_of(-ry * b1), l2 = pair_of(-ry * b2), alpha = pair_of(a.alpha);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = t + i * G;
      if (v * 8 < D) {
        f32x2 dz[4], z[4], g[4];
        if (a.dz) {
          unpack8(reinterpret_cast<const uint4*>(at + plan.dz)[v], dz);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) dz[k] = 0;
        }
        if constexpr (PRE) {
          f32x2 q[4];
          unpack8(reinterpret_cast<const uint4*>(at + plan.z)[v], z);
          unpack8(reinterpret_cast<const uint4*>(at + plan.dh)[v], g);
          gammas(i, q);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (FULL) z[k] = add2(z[k], shift_z);
            z[k] = mul2(z[k], scale_z);
            t1[i][k] = fma2(g[k], z[k], t1[i][k]);
            if constexpr (FULL) {
              t0[i][k] = add2(t0[i][k], g[k]);
              z[k] = fma2(z[k], k2, k1);
            } else {
              z[k] = mul2(z[k], k2);
            }
            dz[k] = add2(dz[k], fma2(mul2(g[k], q[k]), scale_z, z[k]));
          }
        }
        const int64_t c = v * 8;
        if (POST || plan.need_y) unpack8(reinterpret_cast<const uint4*>(at + plan.y)[v], z);
        weights(i, g);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          g[k] = mul2(g[k], dz[k]);
          if (POST || plan.need_y) {
            if constexpr (POST) {
              if constexpr (FULL) z[k] = add2(z[k], shift_y);
              z[k] = mul2(z[k], scale_y);
            }
            s1[i][k] = fma2(dz[k], z[k], s1[i][k]);
          }
          if constexpr (POST) {
            if constexpr (FULL) {
              s0[i][k] = add2(s0[i][k], dz[k]);
              z[k] = fma2(z[k], l2, l1);
            } else {
              z[k] = mul2(z[k], l2);
            }
            g[k] = fma2(g[k], scale_y, z[k]);
          }
          dz[k] = mul2(dz[k], alpha);
        }
        if (dbg_row(a.dx + m * a.lddx + c, c, 8, D, 16)) *reinterpret_cast<uint4*>(a.dx + m * a.lddx + c) = pack8(dz);
        if (dbg_row(a.dy + m * a.lddy + c, c, 8, D, 16)) *reinterpret_cast<uint4*>(a.dy + m * a.lddy + c) = pack8(g);
      }
    }
    row = next;
    next = after;
  }

  // Every copy has landed, each waited for before its row, unless a wait gave
  // up: the last copy into each stage lands before the CTA leaves. (A thread
  // that saw the flag before another has issued fewer; each waits for its own.)
  __syncthreads();
  if (*abort_flag) {
    if (copier)
      for (int i = copied > stages ? copied - stages : 0; i < copied; ++i)
        wait_drain(bar0 + 8u * (i % stages), static_cast<uint32_t>(i / stages) & 1u, wd);
    __syncthreads();
    return;
  }
  // The CTA's partial sums: the groups in order, four sums one after another
  // through [group][2·8·G] in the ring.
  if (!HG_DBG_INDEX(blockIdx.x, kResidualNormPartials) || !HG_DBG_ALIGN(a.partials, 16)) return;
  float* out = a.partials + static_cast<int64_t>(blockIdx.x) * 4 * D;
  auto write_sums = [&](const f32x2 (&s)[NV][4], int which) {
    if constexpr (Cfg::GROUPS > 1) {
      float* all = reinterpret_cast<float*>(ring_smem) + which * (Cfg::THREADS * 8 * NV);
      float* mine = all + group * (NV * 8 * G);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
          *reinterpret_cast<ulonglong2*>(mine + (t + i * G) * 8 + 4 * k) = make_ulonglong2(s[i][2 * k], s[i][2 * k + 1]);
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += Cfg::THREADS) {
        float v = 0.f;
#pragma unroll
        for (int j = 0; j < Cfg::GROUPS; ++j) v += all[j * (NV * 8 * G) + c];
        out[static_cast<int64_t>(which) * D + c] = v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * G) * 8;
        if (c < D) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
            *reinterpret_cast<ulonglong2*>(out + static_cast<int64_t>(which) * D + c + 4 * k) =
                make_ulonglong2(s[i][2 * k], s[i][2 * k + 1]);
        }
      }
    }
  };
  write_sums(s1, 0);
  if constexpr (FULL) write_sums(s0, 1);
  write_sums(t1, 2);
  if constexpr (FULL) write_sums(t0, 3);
}

// What the gradients of a value need of its row: the statistics and the four
// means a1 = mean(g), a2 = mean(g·ẑ) (g = dH·γ), b1 = mean(w·dz),
// b2 = mean(w·dz·ŷ) (w = gate·γ'), a layer norm's a1 and b1 0 for an RMS norm.
struct BackRow {
  float my, ry, mz, rz, a1, a2, b1, b2;
};

__device__ __forceinline__ BackRow back_row(const ResidualNormBackArgs& a, int64_t m) {
  BackRow r{0.f, 1.f, 0.f, 1.f, 0.f, 0.f, 0.f, 0.f};
  if (a.post) r.ry = a.stats[a.M + m];
  if (a.post == HGEMM_NORM_LAYER) r.my = a.stats[m];
  if (a.pre) r.rz = a.stats[3 * a.M + m];
  if (a.pre == HGEMM_NORM_LAYER) r.mz = a.stats[2 * a.M + m];
  return r;
}

// N of a row's values per thread, kThreads apart from column d on, their loads
// all under way at once. KIND: which operands there are.
template <bool POST_, bool PRE_, bool DZ_>
struct BackKind {
  static constexpr bool POST = POST_, PRE = PRE_, DZ = DZ_;
};

template <int N>
struct BackValues {
  float dz[N], dh[N], z[N], y[N], gamma[N], gate[N], w[N];
};

template <typename Kind, int N>
__device__ __forceinline__ BackValues<N> back_values(const ResidualNormBackArgs& a, int64_t m, int64_t d) {
  BackValues<N> v;
  const uint16_t *dz = a.dz + m * a.lddz + d, *dh = a.dh + m * a.lddh + d, *z = a.z + m * a.ldz + d;
  const uint16_t* y = a.y + m * a.ldy + d;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v.dz[i] = Kind::DZ ? half_at(dz, i * kThreads) : 0.f;
    v.dh[i] = Kind::PRE ? half_at(dh, i * kThreads) : 0.f;
    v.z[i] = Kind::PRE ? half_at(z, i * kThreads) : 0.f;
    v.y[i] = half_at(y, i * kThreads);
    v.gamma[i] = Kind::PRE ? half_at(a.pre_gamma, d + i * kThreads) : 0.f;
    v.w[i] = Kind::POST ? half_at(a.post_gamma, d + i * kThreads) : 0.f;
    v.gate[i] = 1.f;
  }
  if (a.gate) {
#pragma unroll
    for (int i = 0; i < N; ++i) v.gate[i] = half_at(a.gate, d + i * kThreads);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) v.w[i] *= v.gate[i];
  return v;
}

// body(values, column of the first, how many) over a row's columns.
template <typename Kind, typename Body>
__device__ __forceinline__ void each_back_value(const ResidualNormBackArgs& a, int64_t m, Body body) {
  constexpr int N = 4;
  int64_t d = threadIdx.x;
  for (; d + (N - 1) * kThreads < a.D; d += N * kThreads) {
    const BackValues<N> v = back_values<Kind, N>(a, m, d);
    body(v, d, std::integral_constant<int, N>{});
  }
  for (; d < a.D; d += kThreads) {
    const BackValues<1> v = back_values<Kind, 1>(a, m, d);
    body(v, d, std::integral_constant<int, 1>{});
  }
}

// dz of one value.
template <typename Kind>
__device__ __forceinline__ float back_dz(const BackRow& r, float dz, float dh, float z, float gamma) {
  return Kind::PRE ? fmaf(r.rz, dh * gamma - r.a1 - (z - r.mz) * r.rz * r.a2, dz) : dz;
}

// Rows that bulk copies cannot describe, or longer than the ring takes: rows
// m0 .. m1-1, whose means the workspace holds. First the four means of every
// row, from the ring's sums ...
template <typename Kind>
__global__ void __launch_bounds__(kThreads) residual_norm_means_kernel(const ResidualNormBackArgs a) {
  __shared__ float s[kThreads / 32][8];
  grid_dependency_wait();
  grid_launch_dependents();
  const float inv_d = 1.f / static_cast<float>(a.D);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int64_t m = a.m0 + blockIdx.x; m < a.m1; m += gridDim.x) {
    if (!HG_DBG_INDEX(m, a.M)) return;
    const BackRow r = back_row(a, m);
    float sums[8] = {};
    each_back_value<Kind>(a, m, [&](const auto& v, int64_t, auto n) {
#pragma unroll
      for (int i = 0; i < decltype(n)::value; ++i) {
        const float zh = (v.z[i] - r.mz) * r.rz, g = v.dh[i] * v.gamma[i];
        const float t = fmaf(g, r.rz, v.dz[i]), wy = (v.y[i] - r.my) * r.ry * v.w[i];
        if (Kind::PRE) {
          sums[0] = fmaf(g, zh, sums[0]);
          sums[3] += g;
        }
        if (Kind::POST) {
          sums[1] = fmaf(wy, t, sums[1]);
          sums[4] = fmaf(v.w[i], t, sums[4]);
        }
        if (Kind::PRE && Kind::POST) {
          sums[2] = fmaf(wy, zh, sums[2]);
          sums[5] = fmaf(v.w[i], zh, sums[5]);
          sums[6] += wy;
          sums[7] += v.w[i];
        }
      }
    });
    const float mine = warp_sums(sums);  // lane l: sum l & 7
    __syncthreads();                     // the row before has been read
    if (lane < 8) s[warp][lane] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sums[j] = 0.f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) sums[j] += s[w][j];
        sums[j] *= inv_d;
      }
      const float a1 = a.pre == HGEMM_NORM_LAYER ? sums[3] : 0.f, a2 = a.pre ? sums[0] : 0.f;
      const float b1 = a.post == HGEMM_NORM_LAYER ? sums[4] - r.rz * (a1 * sums[7] + a2 * sums[5]) : 0.f;
      const float b2 = a.post ? sums[1] - r.rz * (a1 * sums[6] + a2 * sums[2]) : 0.f;
      reinterpret_cast<float4*>(a.means)[m - a.m0] = make_float4(a1, a2, b1, b2);
    }
  }
}

__device__ __forceinline__ BackRow back_row_means(const ResidualNormBackArgs& a, int64_t m) {
  BackRow r = back_row(a, m);
  const float4 v = reinterpret_cast<const float4*>(a.means)[m - a.m0];
  r.a1 = v.x, r.a2 = v.y, r.b1 = v.z, r.b2 = v.w;
  return r;
}

// ... then partial sums down the columns (dX may be dZ and dY may be dH):
// S1 = Σ dz·ŷ, S0 = Σ dz, T1 = Σ dH·ẑ, T0 = Σ dH. Four columns a thread, 32
// apart, which share a row's statistics and means ...
constexpr int kSlices = 80, kSumColumns = 128;
template <typename Kind>
__global__ void __launch_bounds__(kThreads) residual_norm_partials_kernel(const ResidualNormBackArgs a) {
  __shared__ float s[4][8][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, row = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * kSumColumns + c;
  float v[4][4] = {}, gamma[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) gamma[k] = Kind::PRE && d + 32 * k < a.D ? half_at(a.pre_gamma, d + 32 * k) : 0.f;
  for (int64_t m = a.m0 + blockIdx.y * 8 + row; m < a.m1; m += 8 * kSlices) {
    const BackRow r = back_row_means(a, m);
    float dz[4] = {}, dh[4] = {}, z[4] = {}, y[4] = {};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (d + 32 * k < a.D) {
        if (Kind::DZ) dz[k] = half_at(a.dz, m * a.lddz + d + 32 * k);
        if (Kind::PRE) dh[k] = half_at(a.dh, m * a.lddh + d + 32 * k);
        if (Kind::PRE) z[k] = half_at(a.z, m * a.ldz + d + 32 * k);
        y[k] = half_at(a.y, m * a.ldy + d + 32 * k);
      }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float g = back_dz<Kind>(r, dz[k], dh[k], z[k], gamma[k]);
      v[k][0] = fmaf(g, (y[k] - r.my) * r.ry, v[k][0]);
      v[k][1] += g;
      if (Kind::PRE) {
        v[k][2] = fmaf(dh[k], (z[k] - r.mz) * r.rz, v[k][2]);
        v[k][3] += dh[k];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i][row][c] = v[k][i];
    __syncthreads();
    // warp i < 4: the sum i
    if (row < 4 && d + 32 * k < a.D && HG_DBG_INDEX(blockIdx.y, kResidualNormPartials)) {
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += s[row][j][c];
      float* out = a.partials + (static_cast<int64_t>(blockIdx.y) * 4 + row) * a.D + d + 32 * k;
      *out = a.m0 > 0 ? *out + sum : sum;
    }
  }
}

// ... then dX and dY.
template <typename Kind>
__global__ void __launch_bounds__(kThreads) residual_norm_backward_kernel(const ResidualNormBackArgs a) {
  grid_dependency_wait();
  grid_launch_dependents();
  for (int64_t m = a.m0 + blockIdx.x; m < a.m1; m += gridDim.x) {
    if (!HG_DBG_INDEX(m, a.M)) return;
    const BackRow r = back_row_means(a, m);
    each_back_value<Kind>(a, m, [&](const auto& v, int64_t d, auto n) {
#pragma unroll
      for (int i = 0; i < decltype(n)::value; ++i) {
        const int64_t c = d + i * kThreads;
        const float dz = back_dz<Kind>(r, v.dz[i], v.dh[i], v.z[i], v.gamma[i]);
        const float dy =
            Kind::POST ? r.ry * (v.w[i] * dz - r.b1 - (v.y[i] - r.my) * r.ry * r.b2) : v.gate[i] * dz;
        a.dx[m * a.lddx + c] = __half_as_ushort(__float2half_rn(a.alpha * dz));
        a.dy[m * a.lddy + c] = __half_as_ushort(__float2half_rn(dy));
      }
    });
  }
}

// The vectors' gradients from `count` partial sums, in a fixed order: 32
// columns per block, 32 threads down each, whose few loads are all under way at
// once (1000 rows of 1000: 13.4 us for the whole pass with 8 threads and their
// loads one after another, 10.9 this way).
constexpr int kSumThreads = 1024;
__global__ void __launch_bounds__(kSumThreads)
    residual_norm_sums_kernel(const ResidualNormBackArgs a, int count, bool full) {
  constexpr int EACH = (kResidualNormPartials + 31) / 32;
  __shared__ float s[4][32][33];
  grid_dependency_wait();
  grid_launch_dependents();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int64_t d = static_cast<int64_t>(blockIdx.x) * 32 + c;
  float p[EACH][4] = {};
  if (d < a.D) {
#pragma unroll
    for (int i = 0; i < EACH; ++i)
      if (r + 32 * i < count) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (full || j % 2 == 0) p[i][j] = a.partials[(static_cast<int64_t>(r + 32 * i) * 4 + j) * a.D + d];
      }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < EACH; ++i) v += p[i][j];
    s[j][r][c] = v;
  }
  __syncthreads();
  if (r >= 4) return;
  // warp j: the sum j of the 32 columns, then all four by warp 0
  float v = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) v += s[r][i][c];
  s[r][0][c] = v;  // (its own column's sums are read)
  named_bar_sync(1, 128);
  if (r != 0 || d >= a.D || !HG_DBG_INDEX(d, a.D)) return;
  const float s1 = s[0][0][c], s0 = s[1][0][c], t1 = s[2][0][c], t0 = s[3][0][c];
  const float gate = half_or(a.gate, d, 1.f);
  if (a.dgate) a.dgate[d] = a.post ? fmaf(half_at(a.post_gamma, d), s1, half_or(a.post_beta, d, 0.f) * s0) : s1;
  if (a.dpost_gamma) a.dpost_gamma[d] = gate * s1;
  if (a.dpost_beta) a.dpost_beta[d] = gate * s0;
  if (a.dpre_gamma) a.dpre_gamma[d] = t1;
  if (a.dpre_beta) a.dpre_beta[d] = t0;
}

template <int G, int NV>
cudaError_t forward_with(const ResidualNormArgs& a, bool vec, int num_sms, cudaStream_t stream) {
  constexpr int THREADS = kRowsThreads<G>;
  const bool layer = a.post == HGEMM_NORM_LAYER || a.pre == HGEMM_NORM_LAYER;
  const int ahead = G >= 256 || layer ? num_sms * (kResident / G) : 0;
  const int64_t blocks = (a.M + THREADS / G - 1) / (THREADS / G);  // at most 2^31 − 1 rows
  PdlLaunch l(dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, stream);
  return cudaLaunchKernelEx(&l.cfg,
                            vec ? residual_norm_rows_kernel<G, NV, true> : residual_norm_rows_kernel<G, NV, false>, a,
                            ahead);
}

template <int G>
cudaError_t forward_group(const ResidualNormArgs& a, bool vec, int num_sms, cudaStream_t stream) {
  const int64_t nv = (a.D + 8 * G - 1) / (8 * G);
  if (nv <= 1) return forward_with<G, 1>(a, vec, num_sms, stream);
  if (nv <= 2) return forward_with<G, 2>(a, vec, num_sms, stream);
  return forward_with<G, 4>(a, vec, num_sms, stream);
}

template <typename Kernel>
cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !done[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
  }
  return e;
}

template <int G, bool POST, bool PRE, bool FULL>
cudaError_t ring_with(const ResidualNormBackArgs& a, const RingPlan& plan, int grid, cudaStream_t stream) {
  static std::atomic<bool> done[64];
  auto kern = residual_norm_ring_kernel<G, POST, PRE, FULL>;
  const cudaError_t e = allow_smem(kern, RingCfg<G>::SMEM_BYTES, done);
  if (e != cudaSuccess) return e;
  PdlLaunch l(dim3(static_cast<unsigned>(grid)), dim3(RingCfg<G>::THREADS), RingCfg<G>::SMEM_BYTES, stream);
  return cudaLaunchKernelEx(&l.cfg, kern, a, plan);
}

// Whether a call needs the column sums of dz and dH, or a layer norm's means.
bool ring_full(const ResidualNormBackArgs& a) {
  return a.post == HGEMM_NORM_LAYER || a.pre == HGEMM_NORM_LAYER || a.dpost_beta || a.dpre_beta ||
         (a.dgate && a.post_beta);
}

// The ring kernel with G threads per row; *partials: how many it leaves.
template <int G>
cudaError_t ring_group(const ResidualNormBackArgs& a, int num_sms, int* partials, cudaStream_t stream) {
  using Cfg = RingCfg<G>;
  const int64_t want = (a.M + Cfg::GROUPS - 1) / Cfg::GROUPS;
  const int most = num_sms < kResidualNormPartials ? num_sms : kResidualNormPartials;
  const int grid = static_cast<int>(want < most ? want : most);
  RingPlan plan{};
  const uint32_t row = static_cast<uint32_t>(a.D) * 2u;
  plan.need_y = a.post || a.dgate;
  uint32_t at = 0;
  if (a.dz) plan.dz = at, at += row;
  if (a.pre) plan.dh = at, plan.z = at + row, at += 2 * row;
  if (plan.need_y) plan.y = at, at += row;
  plan.stage_bytes = at;
  if (at == 0) plan.stage_bytes = row;  // neither dZ nor dH: nothing is copied
  const uint32_t stages = Cfg::RING_BYTES / (plan.stage_bytes * Cfg::GROUPS);
  plan.stages = static_cast<int>(stages > Cfg::MAX_STAGES ? Cfg::MAX_STAGES : stages);
  plan.empty = at == 0;
  *partials = grid;
  if (!a.post && !a.pre) return ring_with<G, false, false, false>(a, plan, grid, stream);
  if (ring_full(a)) {
    if (!a.post) return ring_with<G, false, true, true>(a, plan, grid, stream);
    return a.pre ? ring_with<G, true, true, true>(a, plan, grid, stream)
                 : ring_with<G, true, false, true>(a, plan, grid, stream);
  }
  if (!a.post) return ring_with<G, false, true, false>(a, plan, grid, stream);
  return a.pre ? ring_with<G, true, true, false>(a, plan, grid, stream)
               : ring_with<G, true, false, false>(a, plan, grid, stream);
}

template <typename Kind>
cudaError_t any_rows_of(const ResidualNormBackArgs& a, cudaStream_t stream) {
  cudaError_t e;
  PdlLaunch r(dim3(rows_grid(a.m1 - a.m0)), dim3(kThreads), 0, stream);
  if ((e = cudaLaunchKernelEx(&r.cfg, residual_norm_means_kernel<Kind>, a)) != cudaSuccess) return e;
  PdlLaunch p(dim3(static_cast<unsigned>((a.D + kSumColumns - 1) / kSumColumns), kSlices), dim3(kThreads), 0, stream);
  if ((e = cudaLaunchKernelEx(&p.cfg, residual_norm_partials_kernel<Kind>, a)) != cudaSuccess) return e;
  return cudaLaunchKernelEx(&r.cfg, residual_norm_backward_kernel<Kind>, a);
}

template <bool POST, bool PRE>
cudaError_t any_rows(const ResidualNormBackArgs& a, cudaStream_t stream) {
  return a.dz ? any_rows_of<BackKind<POST, PRE, true>>(a, stream) : any_rows_of<BackKind<POST, PRE, false>>(a, stream);
}

}  // namespace

cudaError_t launch_residual_norm_forward(const ResidualNormArgs& a, int num_sms, cudaStream_t stream) {
  const bool vec = a.D % 8 == 0 && rows16(a.x, a.ldx) && rows16(a.y, a.ldy) && rows16(a.z, a.ldz) &&
                   rows16(a.h, a.pre ? a.ldh : 8) && rows16(a.gate, 8) && rows16(a.post_gamma, 8) &&
                   rows16(a.post_beta, 8) && rows16(a.pre_gamma, 8) && rows16(a.pre_beta, 8);
  // Enough threads per row to hold it, 32 values each at most (16384 rows of
  // 4096: 128 threads 85 us, 256 threads of 16 values 93, 512 of 8 154; layer
  // norms, 32768 of 2048: 64 threads 91 us, 128 of 16 values 95); when
  // the rows do not fill the GPU, as many as have a piece of it, which is
  // faster for a single row.
  const int64_t each = a.M > 4 * static_cast<int64_t>(num_sms) ? 32 : 8;
  if (a.D <= 32 * each) return forward_group<32>(a, vec, num_sms, stream);
  if (a.D <= 64 * each) return forward_group<64>(a, vec, num_sms, stream);
  if (a.D <= 128 * each) return forward_group<128>(a, vec, num_sms, stream);
  if (a.D <= 256 * each) return forward_group<256>(a, vec, num_sms, stream);
  if (a.D <= 512 * 32) return forward_group<512>(a, vec, num_sms, stream);
  PdlLaunch l(dim3(rows_grid(a.M)), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, residual_norm_long_kernel, a);
}

// Partial sums; the kernels for any row keep theirs in the first kSlices, and
// the rows' means, four values each, in the rest. Where that is little, narrow
// rows, there is room for kMoreRows behind it, since every so many rows are a
// pass of three launches (2^20 rows of 3: 3277 passes without it, 21.3 ms, and
// 213 with it, 4.9 ms; 2^18 of 77: 1.54 and 1.43 ms; 16384 of 65: 95 and 86 us).
constexpr int64_t kMoreRows = 4608;
static int64_t means_rows(int64_t M, int64_t D) {
  const int64_t most = (kResidualNormPartials - kSlices) * ((D + 3) / 4 * 4);
  return M <= most ? most : M <= most + kMoreRows ? M : most + kMoreRows;
}
size_t residual_norm_backward_workspace(int64_t M, int64_t D) {
  return sizeof(float) * 4 * static_cast<size_t>(kSlices * ((D + 3) / 4 * 4) + means_rows(M, D));
}

cudaError_t launch_residual_norm_backward(ResidualNormBackArgs a, int num_sms, cudaStream_t stream) {
  cudaError_t e = cudaSuccess;
  const int64_t most = means_rows(a.M, a.D);
  a.means = a.partials + 4 * kSlices * ((a.D + 3) / 4 * 4);
  int partials = 0;
  const bool ring = a.D % 8 == 0 && a.D <= 8192 && (!a.dz || rows16(a.dz, a.lddz)) &&
                    (!a.pre || (rows16(a.dh, a.lddh) && rows16(a.z, a.ldz) && rows16(a.pre_gamma, 8))) &&
                    rows16(a.y, a.ldy) && rows16(a.dx, a.lddx) && rows16(a.dy, a.lddy) && rows16(a.gate, 8) &&
                    rows16(a.post_gamma, 8);
  if (a.M > 0 && ring) {
    e = a.D <= 512    ? ring_group<32>(a, num_sms, &partials, stream)
        : a.D <= 1024 ? ring_group<64>(a, num_sms, &partials, stream)
        : a.D <= 2048 ? ring_group<128>(a, num_sms, &partials, stream)
        : a.D <= 4096 ? ring_group<256>(a, num_sms, &partials, stream)
                      : ring_group<512>(a, num_sms, &partials, stream);
    if (e != cudaSuccess) return e;
    a.m0 = a.M;
  }
  for (; a.m0 < a.M; a.m0 = a.m1) {
    a.m1 = a.m0 + most < a.M ? a.m0 + most : a.M;
    e = a.post ? (a.pre ? any_rows<true, true>(a, stream) : any_rows<true, false>(a, stream))
               : (a.pre ? any_rows<false, true>(a, stream) : any_rows<false, false>(a, stream));
    if (e != cudaSuccess) return e;
    partials = kSlices;
  }
  if (!a.dgate && !a.dpost_gamma && !a.dpost_beta && !a.dpre_gamma && !a.dpre_beta) return e;
  PdlLaunch l(dim3(static_cast<unsigned>((a.D + 31) / 32)), dim3(kSumThreads), 0, stream);
  return cudaLaunchKernelEx(&l.cfg, residual_norm_sums_kernel, a, partials, !ring || ring_full(a));
}

// The -DHGEMM_DEBUG build's check word of this file (null otherwise).
HG_DEBUG_WORD_ACCESSOR(residual_norm)

}  // namespace hg
